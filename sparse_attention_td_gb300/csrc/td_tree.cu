// td_tree.cu -- attention of a tree of drafted tokens over the decode step's
// cache (contiguous or paged), full or over a persisted index set.
//
// Drafted token t of request b, query head h, KV head g = h / G, context of
// c = seq_lens[b] - n tokens followed by the n drafted ones:
//     S   = C u { c + j : j < n, bit j of mask[b][t] },
//     C   = { 0 .. c - 1 }  or  { idx[b][g][i] in [0, c) },
//     out = sum_{p in S} softmax_p(scale q . K[p]) V[p]        (0 for empty S)
// by an online softmax: running maximum m, denominator l and output o, each
// rescaled by exp(m_old - m_new) when the maximum grows.
//
// All n * G query rows of a (request, KV head) share its K/V rows, so they are
// the M side of two matrix products per tile of 128 tokens: S = Q K^T and
// O += P V, on the tensor cores (tcgen05.mma, 128 query rows; S, P and O in
// tensor memory, K and V tiles in shared memory).  P is rounded to bf16, the
// products' operand type (relative error at most 2^-8, as in the rows themselves);
// S, O, m and l are fp32.  (A second bf16 term of P, 16 bits together, makes P V and
// the softmax longer by more than the loads hide: the cases below 248 -> 270, 241 ->
// 266, 38.4 -> 41.3 and 14.4 -> 15.1 us.  Not taken: the output's own rounding is as
// coarse as one term's.)
//
// What bounds it, measured on GB300 (a copy of the same bytes runs at 6.7 TB/s):
//   reading the cache, once per 128 query rows of a KV head:
//     32 requests of 8K-16K, 8 KV heads, G = 4, 16 nodes, 64-token pages: 248 us, 6.6 TB/s
//     one request of 100K, 32 KV heads, G = 1, 32 nodes:                  242 us, 6.9 TB/s
//     4 x 32K, 8 KV heads, G = 4, 64 nodes (256 rows, two reads): 144-166 us, by where the
//     cache lies, 6.3-7.2 TB/s: twice the time that one read takes
//   launch, first loads and the join, where a step is short:
//     4 x 257-2050, 8 KV heads, G = 8, one node, 16-token pages:  14.6 us
//     (a contiguous cache: 15.0; td_full_attn_select there:       17.9 us)
//     4 x 32K, G = 4, 2048 index entries, 5 nodes:                16.8 us
//     (reads of the same rows alone, call after call:             8.8 us)
//     (the two launches alone, every CTA leaving at once:         4.5 us)
//   copies of single rows, where an index set names them, and the ends of units:
//     32 requests, G = 4, 1024 index entries, 16 nodes:  38.2 us, 3.8 TB/s
// The roles' code together does not fit an SM's instruction cache: on the last of
// these 18% of its requests missed with 100 KB of code and 15% do with 70 KB (waits,
// unit changes and rare cases out of line, loops left rolled, no branches where a
// selection does), which took it from 50 us to 37.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "td_attn_common.cuh"
#include "td_spec.h"

namespace td {
namespace {

constexpr int kTile = 128;                       // tokens per tile, and query rows per unit
constexpr int kHalfBytes = kTile * 128;          // one 64-value half of a tile's rows
constexpr int kTileBytes = 2 * kHalfBytes;       // 128 rows of 128 bf16 values
constexpr int kMaskRing = 8;                     // tiles whose validity masks are alive (see the loader)

// Layout of a CTA.  Shared memory: the Q tile, then the ring of K and V tiles.  Tensor
// memory (512 columns of 32 bits): two S buffers of 128 columns, P over the upper half
// of its S, so S of the next tile is there when a tile's softmax ends, then O.
struct Cfg {
    static constexpr int kSlots = 6;
    static constexpr int kSoftWarps = 4;
    // Warps: softmax, the loader, the MMA issuer, two row finders, copy warps.  Copy
    // warps in the third and fourth sub-partition (warp % 4): their queue of copies
    // slows the other warps there, and the first two have the first 64 rows.
    static constexpr int kLoader = 4, kIssuer = 5, kFinder = 8, kFinders = 2, kCopiers = 4;
    static constexpr int kRowRing = 4;                // tiles whose row lists are alive
    static constexpr int kThreads = 32 * 12;
    // number of a copy warp (6, 7, 10, 11), or -1
    __device__ static int copier(int warp)
    {
        const int w = warp - kSoftWarps;
        return w < 0 || (w & 2) == 0 ? -1 : (w & 1) + (w >> 2) * 2;
    }
    static constexpr size_t kSmem = (size_t)(1 + kSlots) * kTileBytes + 3 * 1024;   // + Extra
    // of tile number g: S and P columns
    __device__ static uint32_t col_s(uint32_t g) { return (g & 1) * 128; }
    __device__ static uint32_t col_p(uint32_t g) { return (g & 1) * 128 + 64; }
    static constexpr uint32_t kColO = 256;
};
constexpr uint32_t kTmemCols = 512;

__device__ __forceinline__ uint32_t smem_of(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint64_t *bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(bar)), "r"(count) : "memory");
}

// One lane of the warp; the MMAs under it issue faster than under lane == 0
// (8 of them in 416 instead of 552 cycles).
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

__device__ __forceinline__ void bar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_of(bar)) : "memory");
}

__device__ __forceinline__ void bar_arrive_n(uint64_t *bar, unsigned n)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(bar)), "r"(n) : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t *bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(bar)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, unsigned parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// What waits look at before they give up: whether another role has, and the tiles done
// by the CTA so far.
struct Progress {
    int gave_up;
    uint32_t tiles;
};

// Waits for the phase of the given parity.  Gives up after `limit` cycles of the SM
// clock without a tile done (a role may have nothing to do for most of a long unit),
// or when another role has (then the CTA leaves as a whole and reports the
// timeout).  Out of line: the roles' code has to stay in the instruction cache.
__device__ __noinline__ bool bar_wait_long(uint32_t bar, unsigned parity, volatile Progress *at, long long limit)
{
    long long t0 = clock64();
    uint32_t tiles = at->tiles;
    for (int polls = 1;; ++polls) {
        if (bar_try(bar, parity))
            return true;
        if ((polls & 63) == 0) {
            if (at->gave_up)
                return false;
            if (at->tiles != tiles) {
                tiles = at->tiles;
                t0 = clock64();
            } else if (clock64() - t0 > limit) {
                at->gave_up = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ bool bar_wait_for(uint64_t *bar, unsigned parity, volatile Progress *at, long long limit)
{
    return bar_try(smem_of(bar), parity) || bar_wait_long(smem_of(bar), parity, at, limit);
}

__device__ __forceinline__ void tma_box(uint32_t dst, const TmaDesc *map, int x, int row, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(row), "r"(smem_of(bar))
        : "memory");
}

// 16 bytes global -> shared, through L2 only; zeros where `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

// The barrier gets this thread's arrival once all of its copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_of(bar)) : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void *p)
{
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Row `tok` of a tile from cache row `row` (none of the cache's `rows`: zeros), by half
// a warp: chunk c at tok * 128 + ((c ^ tok) & 7) * 16 of its half.
__device__ __forceinline__ void copy_row(uint32_t dst, int tok, const uint16_t *src, uint32_t row, uint32_t rows,
                                         int lane)
{
    const int c = lane & 15;
    copy16(dst + (c >> 3) * kHalfBytes + tok * 128 + (((c ^ tok) & 7) << 4),
           src + (size_t)(row < rows ? row : 0) * kHeadDim + c * 8, row < rows);
}

// Shared-memory operand of tcgen05.mma, 128-byte swizzle.  K-major (rows of
// 128 bytes, groups of 8 rows 1024 bytes apart) or, for V, MN-major: 64-value
// blocks of the dims `lead` bytes apart, groups of 8 tokens 1024 bytes apart.
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t lead)   // low word
{
    return ((addr & 0x3ffff) >> 4) | (lead >> 4) << 16;
}
constexpr uint32_t kOperandHigh = 1024 >> 4 | 1u << 14 | 2u << 29;   // high word

// kind::f16, fp32 accumulator, bf16 operands, M = 128; bit 16: B is MN-major.
__host__ __device__ constexpr uint32_t idesc(uint32_t n)
{
    return 1u << 4 | 1u << 7 | 1u << 10 | (n >> 3) << 17 | (128u >> 4) << 24;
}
constexpr uint32_t kIdescV = idesc(128) | 1u << 16;

template <int N> __device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc(N)), "r"((uint32_t)add), "r"(kOperandHigh)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "mov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kIdescV), "r"((uint32_t)add), "r"(kOperandHigh)
        : "memory");
}

// The barrier gets an arrival when every MMA issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_of(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Values that tmem_ld32 loads are used after a tmem_wait_ld and this, which
// keeps their first use behind the wait.
__device__ __forceinline__ void tmem_loaded(uint32_t *r)
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes: thread i gets lane i's values.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
        "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
        "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&x)[4])
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void sts4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void store32(void *p, const uint32_t *x)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 values times f.
__device__ __forceinline__ void scale2(uint32_t *x, float f)
{
    const float2 y = __fmul2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), make_float2(f, f));
    x[0] = __float_as_uint(y.x);
    x[1] = __float_as_uint(y.y);
}

// The same value, which the compiler knows nothing of: a test of it inside a loop
// does not make two loops (the roles' code has to stay in the instruction cache).
template <typename T> __device__ __forceinline__ T opaque(T x)
{
    if constexpr (sizeof(T) == 8)
        asm volatile("" : "+l"(x));
    else
        asm volatile("" : "+r"(x));
    return x;
}

// Block of a request that position p >= 0 lies in: p / page_size by a product.
__device__ __forceinline__ int block_of(const TreeArgs &a, int p)
{
    return (int)((uint64_t)(uint32_t)p * a.page_magic >> a.page_shift);
}

// What a drafted token's V values that are not finite add to an output row that
// sees it, written already, as fp32 partial sums or (part null) as the result.
// Rare; out of line, as is the next one, to keep the roles' code short.
__device__ __noinline__ void add_not_finite(const TreeArgs &a, int b, int h, int pos, float *part, uint16_t *out)
{
    int page = b, r = pos;
    if (a.c.table) {
        const int block = block_of(a, pos);
        page = a.c.table[(size_t)b * a.c.max_blocks + block];
        r = pos - block * a.c.page_size;
    }
    if (page < 0 || page >= a.c.num_pages)
        return;
    const uint16_t *v = a.c.v + (((size_t)page * a.Hkv + h) * a.c.page_size + r) * kHeadDim;
#pragma unroll 1
    for (int k = 0; k < kHeadDim; ++k) {
        if ((v[k] & 0x7f80) != 0x7f80)
            continue;
        const float x = __uint_as_float((uint32_t)v[k] << 16);
        if (part)
            part[k] += x;
        else
            out[k] = (uint16_t)pack_bf16(__uint_as_float((uint32_t)out[k] << 16) + x, 0.0f);
    }
}

// Takes the values that are not finite out of row r of a V tile.
__device__ __noinline__ void clear_not_finite(uint32_t row, int r)
{
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
        uint32_t x[4];
        const uint32_t at = row + (c >> 3) * kHalfBytes + (((c ^ r) & 7) << 4);
        lds_words(at, x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if ((x[k] & 0x7f80u) == 0x7f80u)
                x[k] &= 0xffff0000u;
            if ((x[k] & 0x7f800000u) == 0x7f800000u)
                x[k] &= 0xffffu;
        }
        sts4(at, x[0], x[1], x[2], x[3]);
    }
}

// ---- work: units (request, KV head, block of query rows), each a run of tiles
// of 128 tokens: the context's (or the index set's), then the drafted tokens,
// which share the last context tile where both fit.
struct Work {
    int ctx, nt, tiles, blocks;   // of the current request; tiles 0: no drafted token, no work
    int entries;                  // context tokens, or index entries
    int off;                      // the drafted tokens' first row in the last tile

    // Tokens of tile t; rows behind them are not read.
    __device__ int tokens(int t) const { return t == tiles - 1 ? off + nt : min(kTile, entries - t * kTile); }
};

__device__ __forceinline__ Work work_of(const TreeArgs &a, const TreeLens &len)
{
    Work w;
    w.nt = len.nt;
    w.ctx = len.n - len.nt;
    w.entries = a.idx ? a.top_k : w.ctx;
    const int rest = w.entries & (kTile - 1);
    w.off = rest + w.nt <= kTile ? rest : 0;
    w.tiles = w.nt ? (w.entries >> 7) + (w.off == 0 && rest > 0 ? 1 : 0) + 1 : 0;
    w.blocks = (w.nt * a.G + kTile - 1) / kTile;
    return w;
}

__device__ __forceinline__ Work work_of(const TreeArgs &a, int b, uint32_t &bad)
{
    return work_of(a, tree_lens_of(a.seq_lens, a.tree_lens, b, a.T, a.Nmax, bad));
}

// The first request behind b that has drafted tokens (or the last one) and its
// lengths.  Out of line, once for all roles: their code has to stay in the
// instruction cache.
struct NextRequest {
    TreeLens len;
    int b;
};
__device__ __noinline__ NextRequest next_request(const TreeArgs &a, int b)
{
    NextRequest r;
    uint32_t bad = 0;
#pragma unroll 1
    do {
        r.len = tree_lens_of(a.seq_lens, a.tree_lens, ++b, a.T, a.Nmax, bad);
    } while (r.len.nt == 0 && b + 1 < a.B);
    r.b = b;
    return r;
}

// A CTA's range of tiles, unit after unit: every role of the CTA walks it alike.
struct Walk {
    int left;                     // tiles left of the CTA's range
    int b, h, m, t;               // current request, KV head, row block and first tile
    bool first;                   // the segment starts at the CTA's range start
    Work w;

    __device__ int count() const { return min(left, w.tiles - t); }
    __device__ void next(const TreeArgs &a, int n)
    {
        first = false;
        left -= n;
        t += n;
        if (t < w.tiles || left <= 0)
            return;
        t = 0;
        if (++m < w.blocks)
            return;
        m = 0;
        if (++h < a.Hkv)
            return;
        h = 0;
        const NextRequest r = next_request(a, b);
        b = r.b;
        w = work_of(a, r.len);
    }
    __device__ int rows(const TreeArgs &a) const { return min(w.nt * a.G - m * kTile, kTile); }
};

// Shared memory behind the Q tile and the ring.
//
// Who arrives at a barrier and who waits.  A wait looks at a phase's parity only, so
// each must come when the phase before is over and the one after cannot be:
//   full     a slot's use: the copy warps (as their copies land), or its loader with the
//            boxes' bytes.  The issuer waits for every use in order.  The softmax, at a
//            unit's last tile, for V of tile g: S of g was issued behind P V of g - 3, the
//            use before; the use after needs P V of g, which needs this warp's P.
//   empty    the commit behind the MMAs that read the slot.  The one loader that owns the
//            slot waits for every use in order.
//   rows_there, go, rows_read   a row list, one finder each: written (loaders), then the
//            slots for its K and V free (copy warps), then read (the finder, before it
//            writes the next one there).  Every party waits for every use in order, and
//            the next use needs all of them: its finder all copy warps, these every go,
//            which a loader gives after it has seen rows_there and read rows_valid.
//   q, q_free   as full and empty, per segment, copy warps and issuer.
//   s        S of tile g, every softmax warp waits for every one.  S of g + 2 is issued
//            behind the issuer's wait for p of g, to which every softmax warp arrives.
//   p        all four softmax warps; the issuer waits for every one.
//   o        P V of tile g.  Waited for by the softmax (see o_done) and before S of g + 2
//            (see issue_s): the reasons stand there.
//   drain, done   once, by the issuer.
struct Extra {
    using C = Cfg;
    uint64_t full[C::kSlots], empty[C::kSlots];   // ring: filled, read
    uint64_t q[2], q_free[2];                     // Q of a segment: there, read (by segment parity)
    uint64_t s[2], p[2], o;                       // S there, P there, P V done
    uint64_t rows_there[C::kRowRing], rows_read[C::kRowRing];   // a tile's row list: written, read
    uint64_t go[C::kRowRing][2];                  // the tile's K / V rows may be copied
    uint64_t drain;                               // everything issued is done (a CTA that gave up)
    uint64_t done;                                // everything issued is done
    uint64_t never;                               // nothing arrives (tests of the failure report)
    alignas(16) int rows[C::kRowRing][kTile];     // cache rows of a tile's tokens, -1: none
    uint32_t rows_valid[C::kRowRing][4];          // which tokens have one
    alignas(16) uint32_t valid[kMaskRing][4];     // tokens of a tile that exist
    // Drafted tokens with non-finite V values, by the number of their tile: a warp may
    // look at the next segment's, if it has one or two tiles, while another still
    // reads this one's (behind more, P V has waited for both).
    uint32_t badv[4][4];
    int sums[C::kThreads / 32];
    Walk start;
    uint32_t tmem;
    Progress progress;
    Progress last_waits[C::kThreads / 32];        // of a warp's waits after the CTA gave up
};

// One CTA per SM; each takes an equal, contiguous range of the batch's tiles
// (a range may cover several units and end inside one: those units' partial
// results are joined by tree_join_kernel): the longest request decides nothing, and
// the SMs end together.  Roles: softmax warps (one query row per thread), the
// loader, the row finders and copy warps for tiles that no box holds, and the MMA
// issuer; they meet at barriers in shared memory only.
__global__ void __launch_bounds__(Cfg::kThreads, 1)
tree_attention_kernel(const __grid_constant__ TreeArgs a)
{
    using C = Cfg;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    Extra &x = *reinterpret_cast<Extra *>(sm_raw + (1 + C::kSlots) * kTileBytes);
    static_assert(C::kCopiers == 4, "copy warps' rows of a tile");
    static_assert((1 + C::kSlots) * kTileBytes + sizeof(Extra) <= C::kSmem, "shared memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto bar_wait = [&](uint64_t *bar, unsigned parity, volatile Progress *at) {
        return bar_wait_for(bar, parity, at, a.wait_cycles);
    };
    const uint32_t sm_q = smem_of(sm_raw);        // 1024-byte aligned: nothing static lies before it
    const uint32_t sm_ring = sm_q + kTileBytes;
    volatile Progress *progress = &x.progress;
    if (sm_q & 1023) {            // (cannot be: the swizzled tiles need it)
        if (tid == 0)
            atomicOr(a.status, kFlagWaitTimeout);
        return;
    }

    // ---- what needs no input, while the kernel before this one ends
    if (tid == 32 * C::kLoader) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.box_k) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.box_v) : "memory");
    }
    if (tid == 32 * C::kIssuer) {
        x.progress = Progress{};
        for (int i = 0; i < C::kThreads / 32; ++i)
            x.last_waits[i] = Progress{};
        x.start.left = 0;
        for (int i = 0; i < C::kSlots; ++i) {
            bar_init(&x.full[i], 32 * C::kCopiers);
            bar_init(&x.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&x.q[i], 32 * C::kCopiers);
            bar_init(&x.q_free[i], 1);
            bar_init(&x.s[i], 1);
            bar_init(&x.p[i], 4);
        }
        bar_init(&x.o, 1);
        for (int i = 0; i < C::kRowRing; ++i) {
            bar_init(&x.rows_there[i], 1);
            bar_init(&x.go[i][0], 1);
            bar_init(&x.go[i][1], 1);
            bar_init(&x.rows_read[i], C::kCopiers);
        }
        bar_init(&x.drain, 1);
        bar_init(&x.done, 1);
        bar_init(&x.never, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    {   // the batch's page numbers and index entries into L2, a line per thread of the grid
        const size_t at = ((size_t)blockIdx.x * C::kThreads + tid) * 32;
        if (a.c.table && at < (size_t)a.B * a.c.max_blocks)
            prefetch_l2(a.c.table + at);
        if (a.idx && at < (size_t)a.B * a.Hkv * a.top_k)
            prefetch_l2(a.idx + at);
    }
    // ---- the CTA's range: requests in equal runs per thread, prefix sums.  (The
    // host has made sure that the number of tiles fits 31 bits.)
    {
        const int run = (a.B + C::kThreads - 1) / C::kThreads;
        const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
        uint32_t bad = 0;
        int mine = 0;
        Work w{};
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            w = work_of(a, b, bad);
            mine += w.tiles * w.blocks * a.Hkv;
        }
        if (bad && blockIdx.x == 0)
            atomicOr(a.status, bad);
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, d);
            if (lane >= d)
                inc += y;
        }
        if (lane == 31)
            x.sums[warp] = inc;
        __syncthreads();
        int total = 0, at = inc - mine;
#pragma unroll
        for (int i = 0; i < C::kThreads / 32; ++i) {
            const int y = x.sums[i];
            if (i < warp)
                at += y;
            total += y;
        }
        const int per = (uint32_t)(total + gridDim.x - 1) / gridDim.x;
        const int start = blockIdx.x * per;
        if (start < total && at <= start && start - at < mine) {
            int b = b0;
            if (run > 1) {
#pragma unroll 1
                for (int p = at; b < b1; ++b, at = p) {
                    w = work_of(a, b, bad);
                    p += w.tiles * w.blocks * a.Hkv;
                    if (start < p)
                        break;
                }
            }
            const int unit = (uint32_t)(start - at) / (uint32_t)w.tiles;
            Walk s;
            s.left = min(per, total - start);
            s.b = b;
            s.h = w.blocks == 1 ? unit : unit / w.blocks;
            s.m = unit - s.h * w.blocks;
            s.t = start - at - unit * w.tiles;
            s.first = true;
            s.w = w;
            x.start = s;
        }
        __syncthreads();
        pdl_launch_dependents();
        if (tid == C::kThreads - 1) {
            // The unit that this cut goes through, if it is the unit's first cut.
            JoinPlan j{};
            const int first = x.start.t;
            if (x.start.left > 0 && first > 0 && first <= per) {
                j.rows = x.start.rows(a);
                j.b = x.start.b;
                j.h = x.start.h;
                j.row0 = x.start.m * kTile;
                // the last range that meets the unit
                j.last = (uint32_t)(start - first + x.start.w.tiles - 1) / (uint32_t)per;
                j.late = first < per;
            }
            a.plan[blockIdx.x] = j;
        }
        __syncwarp();
    }
    Walk walk = x.start;
    // Up to 64 query rows per unit: Q has two buffers of 64 rows, and the next
    // segment's comes in during this one.  (The MMA reads 128 rows from either;
    // the rows that are not Q's end in S and O rows that nobody reads.)
    const bool two_q = a.part_rows <= 64;
    uint32_t loaded = 0;          // a loader's ring entries begun
    uint32_t loaded_boxes = 0;    // which of the last ones came as boxes (bit 0: the last)
    uint32_t tmem = 0;
    // Boxes of 8 or 16 rows are more than one warp can issue (80 cycles each).  In full
    // layers the second finder has little to do and loads V, the
    // loader K; the ring's number of slots is even, so each has slots of its own.
    // 32 requests of 8K-16K, G = 4, 16 nodes, one / two loaders: 8-token pages 412 /
    // 258 us, 16: 279 / 253, 32: 251 / 253, 64: 250 / 257 (K then runs ahead of V).
    const bool split = !a.idx && a.box_rows && a.box_rows <= 16;
    const bool loads_v = split && warp == C::kFinder + 1;
    static_assert(C::kSlots % 2 == 0, "slots of K and of V");
    if (warp < C::kSoftWarps || warp == C::kIssuer) {
        // tensor memory for the roles that use it, while the others begin
        if (warp == C::kIssuer) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_of(&x.tmem)),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        tmem_before();
        asm volatile("bar.sync 1, %0;" ::"n"(32 * (C::kSoftWarps + 1)) : "memory");
        tmem_after();
        tmem = x.tmem;
    }

    // The first tiles of a unit, whose tokens all exist, come as boxes of whole rows
    // (of a page) by TMA; the others (ragged end, index set, drafted tokens) row by
    // row by the copy warps.
    auto boxes_of = [&](const Work &w) { return a.idx || !a.box_rows ? 0 : w.ctx >> 7; };
    auto page_of = [&](int b, int p) {
        const int32_t *table = opaque(a.c.table);
        if (!table)
            return b;
        return table[(size_t)b * a.c.max_blocks + block_of(a, p)];
    };
    auto row_of = [&](int h, int pos, int page) {       // -1: no such row
        if (pos < 0 || page < 0 || page >= a.c.num_pages)
            return -1;
        const int in = opaque(a.c.table) ? pos - block_of(a, pos) * a.c.page_size : pos;
        return (page * a.Hkv + h) * a.c.page_size + in;
    };

    if (warp == C::kLoader || loads_v) {
        // ---- loader: waits for the ring's slots, in order, and fills them with boxes
        // or lets the copy warps go.  (Row gathers by TMA took 60 ns per four half
        // rows, 7.7 us a tile.)  Page numbers of the boxes are read 32 at a time, a
        // batch ahead.  The mask ring: the loader is at most kSlots / 2 tiles ahead of
        // the last S = Q K^T, itself at most 2 ahead of the softmax.
        const int shift = a.box_rows ? __ffs(kTile / a.box_rows) - 1 : 0;     // log2(boxes per tile)
        const int batch = 32 >> shift;                                        // tiles per 32 boxes
        auto box_pos = [&](int t, int box) { return t * kTile + box * a.box_rows; };
        const int kv0 = loads_v ? 1 : 0, kv1 = split ? kv0 + 1 : 2;
        uint32_t tile_no = 0, copied = 0, flags = 0;       // tiles; tiles for the copy warps
        bool ok = true;
#pragma unroll 1
        while (ok && walk.left > 0) {
            const int n = walk.count(), boxes = boxes_of(walk.w);
            auto read_pages = [&](int t) {      // of the boxes of tiles t .. t + batch - 1
                const int tile = t + (lane >> shift);
                return tile < boxes ? page_of(walk.b, box_pos(tile, lane & ((1 << shift) - 1))) : 0;
            };
            int first = walk.t, pages = 0, pages2 = 0;
            if (first < boxes) {
                pages = read_pages(first);
                pages2 = read_pages(first + batch);
            }
#pragma unroll 1
            for (int i = 0; i < n; ++i, ++tile_no) {
                const int t = walk.t + i;
                const bool box = t < boxes;
                const uint32_t ring = copied % C::kRowRing;
                int row = 0;                                // of the lane's box
                uint32_t word = kFull;                      // lane < 4: tokens 32 * lane ..
                if (box) {
                    if (t == first + batch) {
                        first = t;
                        pages = pages2;
                        pages2 = read_pages(t + batch);
                    }
                    const int mine = lane & ((1 << shift) - 1);
                    const int page = __shfl_sync(kFull, pages, ((t - first) << shift) + mine);
                    row = row_of(walk.h, box_pos(t, mine), page);
                    const uint32_t there = __ballot_sync(kFull, row >= 0);
                    if (there != kFull) {
                        // a box of a page that does not exist lies behind the cache's rows,
                        // where the map fills with zeros; its tokens do not exist
                        row = row >= 0 ? row : a.c.num_pages * a.Hkv * a.c.page_size;
                        word = 0;
                        for (int k = 0; k < 4; ++k)
                            if (there >> ((32 * (lane & 3) + 8 * k) >> (7 - shift)) & 1u)
                                word |= 0xffu << 8 * k;
                        flags |= kFlagPageOutOfRange;
                    }
                } else {
                    ok = __all_sync(kFull, bar_wait(&x.rows_there[ring], copied / C::kRowRing & 1, progress));
                    if (!ok)
                        break;
                    word = x.rows_valid[ring][lane & 3];
                }
#pragma unroll 1
                for (int kv = kv0; kv < kv1; ++kv) {
                    const uint32_t e = 2 * tile_no + kv, slot = e % C::kSlots, use = e / C::kSlots;
                    if (use > 0)
                        ok = __all_sync(kFull, bar_wait(&x.empty[slot], (use - 1) & 1, progress));
                    if (!ok)
                        break;
                    if (kv == 0 && lane < 4)
                        x.valid[tile_no % kMaskRing][lane] = word;
                    __syncwarp();
                    ++loaded;
                    loaded_boxes = loaded_boxes << 1 | (box ? 1u : 0u);
                    const uint32_t dst = sm_ring + slot * kTileBytes;
                    if (!box) {
                        if (lane == 0)
                            bar_arrive(&x.go[ring][kv]);
                    } else {
                        if (lane == 0) {
                            bar_expect(&x.full[slot], kTileBytes);
                            bar_arrive_n(&x.full[slot], 32 * C::kCopiers - 1);
                        }
                        __syncwarp();
                        const TmaDesc *map = kv ? &a.box_v : &a.box_k;
                        int next = __shfl_sync(kFull, row, 0);
                        uint32_t d = dst;
#pragma unroll 1
                        for (int k = 1; k <= 1 << shift; ++k) {    // (each lane its own: 20% slower)
                            const int r = next;
                            next = __shfl_sync(kFull, row, k & 31);
                            if (elect_one()) {
                                tma_box(d, map, 0, r, &x.full[slot]);
                                tma_box(d + kHalfBytes, map, 64, r, &x.full[slot]);
                            }
                            d += a.box_rows * 128;
                        }
                    }
                    __syncwarp();
                }
                if (!ok)
                    break;
                copied += box ? 0 : 1;
            }
            walk.next(a, n);
        }
        if (flags && lane == 0)
            atomicOr(a.status, flags);
    } else if (warp >= C::kFinder && warp < C::kFinder + C::kFinders) {
        // ---- finders, both of them, or the first where the second loads V: the cache rows
        // of the tiles for the copy warps, as far ahead as there are lists.  (Memory is slow to answer while every SM's
        // ring fills: found by the copy warps themselves, between two tiles, the rows
        // cost 1500 to 3000 cycles a tile.)
        const int me = warp - C::kFinder, finders = split ? 1 : C::kFinders;
        constexpr uint32_t kRing = C::kRowRing;
        uint32_t flags = 0, tile = 0;      // tile: number of the copied tile
        bool ok = true;
#pragma unroll 1
        while (ok && walk.left > 0) {
            const Work &w = walk.w;
            const int n = walk.count();
#pragma unroll 1
            for (int i = max(0, boxes_of(w) - walk.t); i < n; ++i, ++tile) {
                if (finders > 1 && (tile & 1) != (uint32_t)me)
                    continue;
                const int t = walk.t + i, base = t * kTile;
                const bool last = t == w.tiles - 1;
                const int listed = last ? w.off : min(kTile, w.entries - base);   // context entries
                // Loads from valid places whether or not their value counts: no branches.
                // (Plain ones: the kernel before may have written these while this one began.)
                const int32_t *set = a.idx + ((size_t)walk.b * a.Hkv + walk.h) * a.top_k;
                const int32_t *table = a.c.table + (size_t)walk.b * a.c.max_blocks;
                const bool sparse = opaque((int)(a.idx != nullptr)), paged = opaque((int)(a.c.table != nullptr));
                int pos[4], page[4], in[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = base + u * 32 + lane;
                    pos[u] = sparse ? set[min(j, a.top_k - 1)] : j;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int j = u * 32 + lane;
                    if (j >= listed)
                        pos[u] = last && j - w.off < w.nt ? w.ctx + j - w.off : -1;
                    else if (sparse && pos[u] != -1 && (uint32_t)pos[u] >= (uint32_t)w.ctx) {
                        flags |= kFlagIndexOutOfRange;
                        pos[u] = -1;
                    }
                    const int block = paged ? block_of(a, max(pos[u], 0)) : 0;
                    in[u] = pos[u] - block * a.c.page_size;
                    page[u] = paged ? table[block] : walk.b;
                }
                const uint32_t ring = tile % kRing;
                if (tile >= kRing)        // every copy warp has read the list before
                    ok = __all_sync(kFull, bar_wait(&x.rows_read[ring], (tile / kRing - 1) & 1, progress));
                if (!ok)
                    break;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool valid = pos[u] >= 0 && (uint32_t)page[u] < (uint32_t)a.c.num_pages;
                    if (pos[u] >= 0 && !valid)
                        flags |= kFlagPageOutOfRange;
                    const uint32_t there = __ballot_sync(kFull, valid);
                    if (lane == 0)
                        x.rows_valid[ring][u] = there;
                    x.rows[ring][u * 32 + lane] = valid ? (page[u] * a.Hkv + walk.h) * a.c.page_size + in[u] : -1;
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&x.rows_there[ring]);
            }
            walk.next(a, n);
        }
        if (flags)
            atomicOr(a.status, flags);
    } else if (C::copier(warp) >= 0) {
        // ---- copy warps: a segment's Q, then the rows of its tiles that are not
        // boxes, with cp.async, half a warp per 256-byte row; a token that does not
        // exist is filled with zeros (no stale V value meets its zero probability).
        const int me = C::copier(warp);
        constexpr uint32_t kRing = C::kRowRing;
        // No list holds a row outside the cache; one that did would be reported, not followed.
        const uint32_t cache_rows = (uint32_t)(a.c.num_pages * a.Hkv * a.c.page_size);
        bool strange = false;
        uint32_t e = 0, copied = 0;
        bool ok = true;
#pragma unroll 1
        for (uint32_t seg = 0; ok && walk.left > 0; ++seg) {
            const int n = walk.count();
            // Q: its buffer was the last segment's, or with two the one before's.  Rows
            // that are not Q's are left as they are.
            const int last = (int)seg - (two_q ? 2 : 1);
            if (last >= 0)
                ok = __all_sync(kFull, bar_wait(&x.q_free[last & 1], (last >> 1) & 1, progress));
            if (!ok)
                break;
            {
                const int rows = walk.rows(a), row0 = walk.m * kTile;
                const int c = lane & 15;
                const uint16_t *src = a.q + ((size_t)walk.b * a.T * a.Hq + walk.h * a.G) * kHeadDim + c * 8;
                const uint32_t dst = sm_q + (two_q ? seg & 1 : 0) * 64 * 128 + (c >> 3) * kHalfBytes;
#pragma unroll 2
                for (int r = 2 * me + (lane >> 4); r < rows; r += 2 * C::kCopiers) {
                    const int row = row0 + r, tk = row >> a.g_shift, g = row & (a.G - 1);
                    copy16(dst + r * 128 + (((c ^ r) & 7) << 4),
                           src + ((size_t)tk * a.Hq + g) * kHeadDim, true);
                }
                copies_arrive(&x.q[seg & 1]);
            }
#pragma unroll 1
            for (int i = max(0, boxes_of(walk.w) - walk.t); i < n; ++i, ++copied) {
                const uint32_t ring = copied % kRing, phase = copied / kRing & 1;
                const int tokens = walk.w.tokens(walk.t + i);
                // Half a warp takes four neighbouring rows of every 32; their numbers are
                // loaded ahead, as loads from shared memory queue behind the copies.
                const int tok0 = 8 * me + 4 * (lane >> 4);
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv) {
                    ok = __all_sync(kFull, bar_wait(&x.go[ring][kv], phase, progress));
                    if (!ok)
                        break;
                    const uint32_t slot = (e + 2 * i + kv) % C::kSlots;
                    // scores of rows behind the tokens are masked; P V takes tokens by 16
                    const int end = kv ? (tokens + 15) & ~15 : tokens;
                    const uint16_t *src = kv ? a.c.v : a.c.k;
                    const uint32_t dst = sm_ring + slot * kTileBytes;
                    uint32_t rows[4], ahead[4];
                    lds_words(smem_of(&x.rows[ring][tok0]), ahead);
#pragma unroll 1
                    for (int tok = tok0; tok < end; tok += 32) {
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            rows[v] = ahead[v];
                        if (tok + 32 < end)
                            lds_words(smem_of(&x.rows[ring][tok + 32]), ahead);
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (tok + v < end) {
                                copy_row(dst, tok + v, src, rows[v], cache_rows, lane);
                                strange |= rows[v] >= cache_rows && rows[v] != 0xffffffffu;
                            }
                    }
                    copies_arrive(&x.full[slot]);
                }
                __syncwarp();
                if (!ok)
                    break;
                if (lane == 0)
                    bar_arrive(&x.rows_read[ring]);
            }
            e += 2 * n;
            walk.next(a, n);
        }
        if (strange)
            atomicOr(a.status, kFlagPageOutOfRange);
    } else if (warp == C::kIssuer) {
        // ---- MMA issue, by one thread: S of tile j + 1 before P V of tile j, so the
        // tensor cores work while the softmax does.
        if (elect_one()) {
            uint32_t e = 0;              // ring entry of the segment's first K tile
            uint32_t tiles = 0;          // tiles of earlier segments
            uint32_t seg = 0;            // segments begun
            bool ok = true;
            // Rows copied by cp.async are read by the MMA through the async proxy; boxes
            // come through it and need no fence.
            auto proxy_fence = [] { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); };
            auto wait_full = [&](uint32_t entry, bool copied) {
                ok = ok && bar_wait(&x.full[entry % C::kSlots], (entry / C::kSlots) & 1, progress);
                if (copied)
                    proxy_fence();
                return ok;
            };
            auto wait_bar = [&](uint64_t *bar, uint32_t phase) {
                ok = ok && bar_wait(bar, phase & 1, progress);
                tmem_after();
                return ok;
            };
#pragma unroll 1
            for (; ok && walk.left > 0; ++seg) {
                const int n = walk.count();
                const uint32_t q = operand(sm_q + (two_q ? seg & 1 : 0) * 64 * 128, 16);
                auto issue_s = [&](int j) {
                    const uint32_t slot = (e + 2 * j) % C::kSlots, g = tiles + j;
                    const uint32_t k = operand(sm_ring + slot * kTileBytes, 16);
                    // P V of tile g - 2 has read the P that goes next.  (j = 0: its softmax has
                    // waited for that before it handed over P of tile g - 1.  The phase before is
                    // over by then, and P V of tile g - 1 is issued later: no phase is missed.)
                    if (j >= 1 && g >= 2)
                        wait_bar(&x.o, g - 2);
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t o = (s >> 2) * kHalfBytes + (s & 3) * 32;
                        mma_ss<kTile>(tmem + C::col_s(g), q + (o >> 4), k + (o >> 4), s > 0);
                    }
                    mma_commit(&x.s[g & 1]);
                    mma_commit(&x.empty[slot]);
                    if (j == n - 1)
                        mma_commit(&x.q_free[seg & 1]);   // the segment's Q has been read
                };
                const int boxes = boxes_of(walk.w) - walk.t;     // tiles before this one are boxes
                wait_bar(&x.q[seg & 1], seg >> 1);
                proxy_fence();
                if (!wait_full(e, boxes <= 0))
                    break;
                issue_s(0);
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    if (j + 1 < n) {
                        if (!wait_full(e + 2 * (j + 1), j + 1 >= boxes))
                            break;
                        issue_s(j + 1);
                    }
                    const uint32_t entry = e + 2 * j + 1, slot = entry % C::kSlots, g = tiles + j;
                    if (!wait_full(entry, j >= boxes))
                        break;
                    const uint32_t v = operand(sm_ring + slot * kTileBytes, kHalfBytes);
                    const int tokens = walk.w.tokens(walk.t + j);    // by 16, as far as there are any
                    if (!wait_bar(&x.p[g & 1], g >> 1))
                        break;
#pragma unroll
                    for (int s = 0; s < kTile / 16; ++s)
                        if (s * 16 < tokens)
                            mma_ts(tmem + C::kColO, tmem + C::col_p(g) + s * 8, v + (s * 16 * 128 >> 4),
                                   j > 0 || s > 0);
                    mma_commit(&x.o);
                    mma_commit(&x.empty[slot]);
                    progress->tiles = g + 1;
                }
                tiles += n;
                e += 2 * n;
                walk.next(a, n);
            }
            // Nobody waits for the last commits to the ring's slots and Q: no arrival of
            // theirs may be left when the CTA ends.
            mma_commit(&x.done);
            bar_wait(&x.done, 0, progress);
        }
        __syncwarp();
    } else {
        // ---- softmax: thread r owns query row r of the unit
        const int r = warp * 32 + lane;                       // also the TMEM lane
        const uint32_t lanes = (uint32_t)warp << 21;          // this warp's TMEM lanes
        const float sl2 = a.scale * kLog2e;
        uint32_t count = 0;                                   // tiles done
        bool ok = true;
#pragma unroll 1
        while (ok && walk.left > 0) {
            const int n = walk.count();
            const int b = walk.b, h = walk.h;
            const int row0 = walk.m * kTile;                   // first query row of the unit
            const int total_rows = walk.w.nt * a.G;
            const size_t q0 = (size_t)b * a.T * a.Hq + h * a.G;
            const int row = row0 + r;
            const int tok = row >> a.g_shift;                  // drafted token of this row
            const bool live = row < total_rows;
            const bool warp_live = row0 + warp * 32 < total_rows;
            float mref = -CUDART_INF_F, l = 0.0f;
            uint32_t sees[4] = {0, 0, 0, 0};
            const bool has_tree = walk.t + n == walk.w.tiles;
            if (has_tree && live) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    if (a.mask)
                        sees[w] = w < a.W ? a.mask[((size_t)b * a.T + tok) * a.W + w] : 0u;
                    else
                        sees[w] = tok >= 32 * w + 31 ? 0xffffffffu
                                  : tok >= 32 * w   ? 0xffffffffu >> (31 - (tok & 31))
                                                    : 0u;
                }
            }
#pragma unroll 1
            for (int j = 0; j < n; ++j, ++count) {
                const bool tree = walk.t + j == walk.w.tiles - 1;
                // P V of the tile before is done: waited for to rescale O, and at the last
                // tile.  (P V of the tile before that was done when S of this one was
                // issued, so no phase is missed.)  Both waits come before P of this tile is
                // handed over, behind which its P V may end and the phase of the one before
                // be past.
                bool waited = j == 0;
                auto o_done = [&]() {
                    if (!waited)
                        ok = __all_sync(kFull, bar_wait(&x.o, (count - 1) & 1, progress));
                    waited = true;
                };
                ok = __all_sync(kFull, bar_wait(a.wait_test ? &x.never : &x.s[count & 1],
                                                a.wait_test ? 0 : count >> 1 & 1, progress));
                if (!ok)
                    break;
                tmem_after();
                if (tree) {
                    // the last tile's bits: its context tokens, then the drafted ones
                    uint64_t lo = sees[0] | (uint64_t)sees[1] << 32, hi = sees[2] | (uint64_t)sees[3] << 32;
                    const int off = walk.w.off;
                    const uint64_t below = (1ull << (off & 63)) - 1;
                    hi = off >= 64 ? lo << (off & 63) | below : off > 0 ? hi << off | lo >> (64 - off) : hi;
                    lo = off >= 64 ? ~0ull : lo << off | below;
                    sees[0] = (uint32_t)lo;
                    sees[1] = (uint32_t)(lo >> 32);
                    sees[2] = (uint32_t)hi;
                    sees[3] = (uint32_t)(hi >> 32);
                    // A V value that is not finite must not meet the zero
                    // probabilities of rows that do not see its token: such values
                    // leave the tile here and join the rows that do see it below.
                    const uint32_t entry = 2 * count + 1;
                    ok = __all_sync(kFull, bar_wait(&x.full[entry % C::kSlots],
                                                    (entry / C::kSlots) & 1, progress));
                    if (!ok)
                        break;
                    const uint32_t v = sm_ring + entry % C::kSlots * kTileBytes + r * 128;
                    bool any = false;
                    if (r >= walk.w.off && r < walk.w.off + walk.w.nt) {
                        // largest magnitude bits of the row's even and odd values
                        uint32_t top = 0;
#pragma unroll 8
                        for (int c = 0; c < 16; ++c) {
                            uint32_t y4[4];
                            lds_words(v + (c >> 3) * kHalfBytes + (((c ^ r) & 7) << 4), y4);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                top = __vmaxu2(top, y4[k] & 0x7fff7fffu);
                        }
                        any = (top & 0xffffu) >= 0x7f80u || top >= 0x7f800000u;
                    }
                    const uint32_t bits = __ballot_sync(kFull, any);
                    if (lane == 0)
                        x.badv[count & 3][warp] = bits;
                    if (bits) {
                        if (any)
                            clear_not_finite(v, r);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                }
                if (warp_live) {
                    // The row's scores pass through 64 registers, in blocks of 64
                    // tokens: every block once for the maximum, then the last block
                    // from the registers and the others again for the exponentials.
                    // A loop that stays rolled: with the step unrolled over 128
                    // registers the roles' code no longer fitted the instruction
                    // cache (100K: 261 us against 314).
                    const uint32_t at = tmem + C::col_s(count) + lanes;
                    uint32_t seen[4];                 // of the tile's tokens, 32 a word
                    lds_words(smem_of(x.valid[count % kMaskRing]), seen);
                    if (tree) {
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            seen[w] &= sees[w];
                    }
                    float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                    float2 off2 = make_float2(0.0f, 0.0f);
                    float2 sum[2] = {off2, off2};
                    // passes: block 0 (maximum), block 1 (maximum, probabilities), block 0
                    // (probabilities); with one block of tokens both in one
                    const int blocks = walk.w.tokens(walk.t + j) > 64 ? 2 : 1;
#pragma unroll 1
                    for (int pass = 0; pass < 2 * blocks - 1; ++pass) {
                        const int block = blocks > 1 ? pass & 1 : 0;
                        const uint32_t w0 = block > 0 ? seen[2] : seen[0], w1 = block > 0 ? seen[3] : seen[1];
                        float s[64];
                        __syncwarp();
                        tmem_ld32(at + 64 * block, reinterpret_cast<uint32_t *>(s));
                        tmem_ld32(at + 64 * block + 32, reinterpret_cast<uint32_t *>(s) + 32);
                        tmem_wait_ld();
                        tmem_loaded(reinterpret_cast<uint32_t *>(s));
                        tmem_loaded(reinterpret_cast<uint32_t *>(s) + 32);
                        if ((w0 & w1) != kFull) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                if (!(w0 >> k & 1u))
                                    s[k] = -CUDART_INF_F;
                                if (!(w1 >> k & 1u))
                                    s[32 + k] = -CUDART_INF_F;
                            }
                        }
                        if (pass < blocks) {
#pragma unroll
                            for (int k = 0; k < 64; k += 2)
                                mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], s[k], s[k + 1]);
                        }
                        if (pass == blocks - 1) {
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                            if (mref == -CUDART_INF_F)
                                mref = top;          // nothing summed so far: l = 0 and O = 0
                            // The running maximum lags until a row exceeds it by 2^8: the
                            // probabilities stay below 2^8 and the rescaling of O is rare.
                            const bool grow = j > 0 && top > mref + 8.0f;
                            if (__any_sync(kFull, grow)) {
                                o_done();
                                if (!ok)
                                    break;
                                tmem_after();
                                const float mn = grow ? top : mref;
                                const float f = grow ? ex2(mref - mn) : 1.0f;
                                mref = mn;
                                l *= f;
                                const uint32_t o = tmem + C::kColO + lanes;
#pragma unroll 1
                                for (int c = 0; c < 4; ++c) {
                                    uint32_t ov[32];
                                    tmem_ld32(o + 32 * c, ov);
                                    tmem_wait_ld();
                                    tmem_loaded(ov);
#pragma unroll
                                    for (int k = 0; k < 32; k += 2)
                                        scale2(ov + k, f);
                                    tmem_st32(o + 32 * c, ov);
                                }
                            }
                            const float off = mref == -CUDART_INF_F ? 0.0f : -mref;
                            off2 = make_float2(off, off);
                        }
                        if (pass >= blocks - 1) {
                            const float2 sl22 = make_float2(sl2, sl2);
                            uint32_t p[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const float2 z = __ffma2_rn(make_float2(s[2 * k], s[2 * k + 1]), sl22, off2);
                                const float2 e = make_float2(ex2(z.x), ex2(z.y));
                                sum[k & 1] = __fadd2_rn(sum[k & 1], e);
                                p[k] = pack_bf16(e.x, e.y);
                            }
                            // (over scores of this or a later block, which have been read)
                            tmem_st32(tmem + C::col_p(count) + lanes + 32 * block, p);
                        }
                    }
                    if (!ok)
                        break;
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    tmem_wait_st();
                }
                if (j == n - 1)
                    o_done();
                if (!ok)
                    break;
                tmem_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&x.p[count & 1]);
            }
            if (!ok)
                break;
            // ---- the segment's result
            ok = __all_sync(kFull, bar_wait(&x.o, (count - 1) & 1, progress));
            if (!ok)
                break;
            tmem_after();
            if (warp_live) {
                const bool whole = n == walk.w.tiles;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const int part = 2 * blockIdx.x + (walk.first ? 0 : 1);
                const size_t prow = (size_t)part * a.part_rows + r;
                uint16_t *out = a.out + (q0 + (size_t)tok * a.Hq + (row & (a.G - 1))) * kHeadDim;
                float *part_o = a.part_o + prow * kHeadDim;
                const uint32_t o = tmem + C::kColO + lanes;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t ov[32];
                    tmem_ld32(o + 32 * c, ov);
                    tmem_wait_ld();
                    tmem_loaded(ov);
                    if (live && whole) {
                        uint16_t *dst = out + 32 * c;
                        uint32_t y[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            scale2(ov + 2 * k, inv);
                            y[k] = pack_bf16(__uint_as_float(ov[2 * k]), __uint_as_float(ov[2 * k + 1]));
                        }
                        const uint4 *v = reinterpret_cast<const uint4 *>(y);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            reinterpret_cast<uint4 *>(dst)[k] = v[k];
                    } else if (live) {
                        float *dst = part_o + 32 * c;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            store32(dst + 8 * k, ov + 8 * k);
                    }
                    __syncwarp();
                }
                if (!whole && live) {
                    a.part_m[prow] = mref;
                    a.part_l[prow] = l;
                }
                if (has_tree && live) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t bad = x.badv[(count - 1) & 3][w] & sees[w];
                        for (; bad; bad &= bad - 1)
                            add_not_finite(a, b, h, walk.w.ctx + 32 * w + __ffs(bad) - 1 - walk.w.off,
                                           whole ? nullptr : part_o, out);
                    }
                }
                __syncwarp();
                tmem_before();
            }
            __syncwarp();
            walk.next(a, n);
        }
    }
    tmem_before();
    __syncthreads();
    if (x.progress.gave_up) {
        // A wait gave up: leave no copy and no MMA in flight.  Of the boxes the last
        // entries of a loader's slots can be; what was issued does complete, and these
        // waits have the default limit.
        constexpr long long kLimit = 2000000000ll;
        volatile Progress *own = &x.last_waits[warp];
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (warp == C::kLoader || loads_v) {
            const uint32_t slots = split ? C::kSlots / 2 : C::kSlots;
            for (uint32_t n = loaded > slots ? loaded - slots : 0; n < loaded; ++n) {
                const uint32_t e = split ? 2 * n + (loads_v ? 1 : 0) : n;
                if (loaded_boxes >> (loaded - 1 - n) & 1)
                    bar_wait_for(&x.full[e % C::kSlots], (e / C::kSlots) & 1, own, kLimit);
            }
        } else if (warp == C::kIssuer && elect_one()) {      // (the lane that issued them)
            mma_commit(&x.drain);
            bar_wait_for(&x.drain, 0, own, kLimit);
        }
        __syncthreads();
    }
    if (tid == 0 && x.progress.gave_up)
        atomicOr(a.status, kFlagWaitTimeout);
    if (warp == C::kIssuer) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
    }
}

// Joins the parts of the units that several CTAs shared.  Block x belongs to
// the cut at the start of CTA x + 1's range, which left a plan of the unit that
// it goes through (rows 0: none, or another cut's unit).  A warp per query row:
// o = sum_s o_s 2^(m_s - m) / sum_s l_s 2^(m_s - m).
constexpr int kJoinWarps = 4;

__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ JoinArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.x + 1;
    const JoinPlan j = a.plan[c];
    const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
    if (r >= j.rows)
        return;
    // part s of the unit: CTA c - 1 + s's; its second one where the unit starts inside its range
    auto part_row = [&](int s) {
        return (size_t)(2 * (c - 1 + s) + (s == 0 && j.late ? 1 : 0)) * a.part_rows + r;
    };
    auto not_finite = [](float v) { return fabsf(v) < CUDART_INF_F ? 0.0f : v; };
    const int parts = j.last - c + 2;
    constexpr int kAhead = 8;
    float top = -CUDART_INF_F, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < parts; s0 += kAhead) {
        float ms[kAhead], ls[kAhead];
        float4 x[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            ms[u] = -CUDART_INF_F;
            ls[u] = 0.0f;
            if (s0 + u < parts) {
                const size_t p = part_row(s0 + u);
                ms[u] = a.part_m[p];
                ls[u] = a.part_l[p];
                x[u] = *reinterpret_cast<const float4 *>(a.part_o + p * kHeadDim + lane * 4);
            }
        }
        float mn = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            mn = fmaxf(mn, ms[u]);
        const float keep = safe_exp2_diff(top, mn);
        l *= keep;
        o.x *= keep;
        o.y *= keep;
        o.z *= keep;
        o.w *= keep;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const float f = safe_exp2_diff(ms[u], mn);
            // an empty part has nothing to add; one whose scores are all NaN has no maximum
            if (f != 0.0f || ls[u] != ls[u]) {
                l += ls[u] * f;
                o.x += x[u].x * f;
                o.y += x[u].y * f;
                o.z += x[u].z * f;
                o.w += x[u].w * f;
            } else if (ls[u] != 0.0f) {
                // a weight too small for fp32 is not zero: what is not finite stays so
                o.x += not_finite(x[u].x);
                o.y += not_finite(x[u].y);
                o.z += not_finite(x[u].z);
                o.w += not_finite(x[u].w);
            }
        }
        top = mn;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int row = j.row0 + r;
    uint2 y;
    y.x = pack_bf16(o.x * inv, o.y * inv);
    y.y = pack_bf16(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(
        a.out + (((size_t)j.b * a.T + row / a.G) * a.Hq + j.h * a.G + row % a.G) * kHeadDim + lane * 4) = y;
}

}  // namespace

cudaError_t launch_tree_attention(const TreeArgs &a, int sms, cudaStream_t stream)
{
    using C = Cfg;
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !ready[dev]) {
            err = cudaFuncSetAttribute(tree_attention_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
            if (err != cudaSuccess)
                return err;
            if (dev >= 0 && dev < 64)
                ready[dev] = true;
        }
    }
    const int ctas = sms < kMaxTreeCtas ? sms : kMaxTreeCtas;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    err = cudaLaunchKernelEx(&cfg, tree_attention_kernel, a);
    if (err != cudaSuccess || ctas < 2)
        return err;
    cfg.gridDim = dim3(ctas - 1, (a.part_rows + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    const JoinArgs j{a.plan, a.part_m, a.part_l, a.part_o, a.out, a.T, a.Hq, a.G, a.part_rows};
    return cudaLaunchKernelEx(&cfg, tree_join_kernel, j);
}

}  // namespace td
