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
// O += P V, on the tensor cores (tcgen05.mma, 128 x 128 tiles; S, P and O in
// tensor memory, K and V tiles in shared memory).  A K/V byte then takes part
// in up to 128 (one row tile) or 256 (two) multiply-adds, and the layer is
// bound by reading the cache.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "td_attn_common.cuh"
#include "td_spec.h"

namespace td {
namespace {

constexpr int kTile = 128;                       // tokens per tile, and query rows per row tile
constexpr int kHalfBytes = kTile * 128;          // one 64-value half of a tile's rows
constexpr int kTileBytes = 2 * kHalfBytes;       // 128 rows of 128 bf16 values
constexpr int kMaskRing = 8;                     // tiles whose validity masks are alive (see producer)
constexpr uint64_t kTreeWaitNs = 1000000000ull;  // a wait gives up after 1 s

// Shared memory: Q row tiles, then the ring of K and V tiles.
template <int MT> struct Cfg {
    static constexpr int kSlots = MT == 1 ? 6 : 5;
    static constexpr int kSoftWarps = 4 * MT;
    static constexpr int kThreads = 32 * (kSoftWarps + 2);
    static constexpr size_t kSmem = (size_t)(MT + kSlots) * kTileBytes + 1024;
};
// Tensor memory columns (32-bit): two S tiles (P overwrites the lower half of
// its S), then the O tiles.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;

__device__ __forceinline__ uint32_t smem_of(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void bar_init(uint64_t *bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_of(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_of(bar)) : "memory");
}

__device__ __forceinline__ void bar_expect(uint64_t *bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_of(bar)),
                 "r"(bytes)
                 : "memory");
}

// Waits for the phase of the given parity.  Gives up after kTreeWaitNs, or when
// another role has (then the CTA leaves as a whole and reports the timeout).
__device__ __forceinline__ bool bar_wait(uint64_t *bar, unsigned parity, volatile int *gave_up)
{
    const uint32_t addr = smem_of(bar);
    uint64_t t0 = 0;
    for (int polls = 0;; ++polls) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity)
            : "memory");
        if (done)
            return true;
        if ((polls & 15) == 15) {
            uint64_t t;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
            if (t0 == 0)
                t0 = t;
            if (*gave_up)
                return false;
            if (t - t0 > kTreeWaitNs) {
                *gave_up = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ void tma_box(uint32_t dst, const TmaDesc *map, int x, int row, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(row), "r"(smem_of(bar))
        : "memory");
}

__device__ __forceinline__ void tma_rows4(uint32_t dst, const TmaDesc *map, int x, const int (&r)[4],
                                          uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(smem_of(bar))
        : "memory");
}

// Shared-memory operand of tcgen05.mma, 128-byte swizzle.  K-major (rows of
// 128 bytes, groups of 8 rows 1024 bytes apart) or, for V, MN-major: 64-value
// blocks of the dims `lead` bytes apart, groups of 8 tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | (uint64_t)(lead >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// kind::f16, fp32 accumulator, bf16 operands, M = N = 128; bit 16: B is MN-major.
constexpr uint32_t kIdesc = 1u << 4 | 1u << 7 | 1u << 10 | (128u >> 3) << 17 | (128u >> 4) << 24;
constexpr uint32_t kIdescV = kIdesc | 1u << 16;

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(kIdesc), "r"((uint32_t)add)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(kIdescV), "r"((uint32_t)add)
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

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void lds4(uint32_t addr, uint32_t (&x)[4])
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

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ---- work: units (request, KV head, block of query rows), each a run of
// tiles: the context's (or the index set's), then one tile of drafted tokens.
struct Work {
    int ctx, nt, tiles, blocks;   // of the current request; tiles 0: no drafted token, no work
};

template <int MT>
__device__ __forceinline__ Work work_of(const TreeArgs &a, int b, uint32_t &bad)
{
    const TreeLens len = tree_lens_of(a.seq_lens, a.tree_lens, b, a.T, a.Nmax, bad);
    Work w;
    w.nt = len.nt;
    w.ctx = len.n - len.nt;
    const int entries = a.idx ? a.top_k : w.ctx;
    w.tiles = w.nt ? (int)(((long long)entries + kTile - 1) / kTile) + 1 : 0;
    w.blocks = (w.nt * a.G + MT * kTile - 1) / (MT * kTile);
    return w;
}

// A CTA's range of tiles, unit after unit: every role of the CTA walks it alike.
template <int MT> struct Walk {
    const TreeArgs &a;
    long long left;
    int b, h, m, t;               // current request, KV head, row block and first tile
    bool first;                   // the segment starts at the CTA's range start
    Work w;

    __device__ Walk(const TreeArgs &args, int b0, long long off, long long n)
        : a(args), left(n), b(b0), first(true)
    {
        uint32_t bad = 0;
        w = work_of<MT>(a, b, bad);
        const long long unit = off / w.tiles;
        t = (int)(off % w.tiles);
        h = (int)(unit / w.blocks);
        m = (int)(unit % w.blocks);
    }
    __device__ int count() const { return (int)min(left, (long long)(w.tiles - t)); }
    __device__ void next(int n)
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
        uint32_t bad = 0;
        do {
            w = work_of<MT>(a, ++b, bad);
        } while (w.tiles == 0 && b + 1 < a.B);
    }
    __device__ int rows() const { return min(w.nt * a.G - m * MT * kTile, MT * kTile); }
};

// One CTA per SM; each takes an equal, contiguous range of the batch's tiles
// (a range may cover several units and end inside one: those units' partial
// results are joined by tree_join_kernel).  Roles: 4 * MT softmax warps (one
// query row per thread), a warp that fills the ring, a warp that issues MMAs.
template <int MT>
__global__ void __launch_bounds__(Cfg<MT>::kThreads, 1)
tree_attention_kernel(const __grid_constant__ TreeArgs a)
{
    using C = Cfg<MT>;
    extern __shared__ unsigned char sm_raw[];
    __shared__ __align__(8) uint64_t bar_full[C::kSlots], bar_empty[C::kSlots];
    __shared__ __align__(8) uint64_t bar_q[MT], bar_s[2], bar_p[2], bar_o[MT], bar_scan, bar_drain;
    __shared__ uint32_t sm_valid[kMaskRing][4];   // tokens of a tile that exist
    __shared__ uint32_t sm_badv[MT][4];           // drafted tokens with non-finite V values
    __shared__ long long sm_scan[C::kThreads / 32];
    __shared__ long long sm_off;
    __shared__ int sm_b0;
    __shared__ uint32_t sm_tmem;
    __shared__ int sm_gave_up;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sm_q = (smem_of(sm_raw) + 1023) & ~1023u;
    const uint32_t sm_ring = sm_q + MT * kTileBytes;
    volatile int *gave_up = &sm_gave_up;

    // ---- the CTA's range: requests in equal runs per thread, prefix sums
    long long start, end;
    {
        const int run = (a.B + C::kThreads - 1) / C::kThreads;
        const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
        uint32_t bad = 0;
        long long mine = 0;
        for (int b = b0; b < b1; ++b) {
            const Work w = work_of<MT>(a, b, bad);
            mine += (long long)w.tiles * w.blocks * a.Hkv;
        }
        if (bad && blockIdx.x == 0)
            atomicOr(a.status, bad);
        long long inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long y = __shfl_up_sync(kFull, inc, d);
            if (lane >= d)
                inc += y;
        }
        if (lane == 31)
            sm_scan[warp] = inc;
        if (tid == 0) {
            sm_gave_up = 0;
            for (int i = 0; i < C::kSlots; ++i) {
                bar_init(&bar_full[i], 1);
                bar_init(&bar_empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                bar_init(&bar_s[i], 1);
                bar_init(&bar_p[i], 4);
            }
            for (int i = 0; i < MT; ++i) {
                bar_init(&bar_q[i], 4);
                bar_init(&bar_o[i], 1);
            }
            bar_init(&bar_scan, 4);
            bar_init(&bar_drain, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncthreads();
        long long total = 0, at = inc - mine;
        for (int i = 0; i < C::kThreads / 32; ++i) {
            if (i < warp)
                at += sm_scan[i];
            total += sm_scan[i];
        }
        const long long per = (total + gridDim.x - 1) / gridDim.x;
        start = blockIdx.x * per;
        end = min(start + per, total);
        if (blockIdx.x == 0) {
            long long p = at;
            for (int b = b0; b < b1; ++b) {
                const Work w = work_of<MT>(a, b, bad);
                a.prefix[b] = p;
                p += (long long)w.tiles * w.blocks * a.Hkv;
            }
            if (tid == 0)
                a.prefix[a.B] = total;
        }
        pdl_launch_dependents();
        if (start >= end)
            return;
        if (at <= start && start < at + mine) {
            long long p = at;
            for (int b = b0; b < b1; ++b) {
                const Work w = work_of<MT>(a, b, bad);
                const long long n = (long long)w.tiles * w.blocks * a.Hkv;
                if (start < p + n) {
                    sm_b0 = b;
                    sm_off = start - p;
                    break;
                }
                p += n;
            }
        }
        __syncwarp();
        if (warp == C::kSoftWarps + 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_of(&sm_tmem)),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
        tmem_before();
        __syncthreads();
        tmem_after();
    }
    const uint32_t tmem = sm_tmem;
    Walk<MT> walk(a, sm_b0, sm_off, end - start);

    if (warp == C::kSoftWarps) {
        // ---- producer: K then V tile of every tile in turn, into the ring.
        // A tile whose tokens all exist comes as boxes of whole rows (of a page);
        // any other (ragged end, index set, drafted tokens, a bad page) row by
        // row, four per copy, where a token that does not exist reads the zero
        // row past the map: its V row is then 0, and the validity mask keeps its
        // score out.  The mask ring: the producer is at most kSlots / 2 tiles
        // ahead of the last S = Q K^T, itself at most 2 ahead of the softmax.
        uint32_t e = 0, tile_no = 0;
        bool ok = true;
        while (ok && walk.left > 0) {
            const int n = walk.count();
            const int h = walk.h, b = walk.b;
            for (int i = 0; ok && i < n; ++i, ++tile_no) {
                const int t = walk.t + i;
                const bool tree = t == walk.w.tiles - 1;
                const int base = t * kTile;
                int rows[4];
                int box = -1;               // this lane's box row
                uint32_t flags = 0;
                bool boxes = false;
                if (!tree && !a.idx && a.box_rows && base + kTile <= walk.w.ctx) {
                    const int nbox = kTile / a.box_rows;
                    if (lane < nbox) {
                        const int p = base + lane * a.box_rows;
                        int page = b, r = p;
                        if (a.c.table) {
                            page = a.c.table[(size_t)b * a.c.max_blocks + p / a.c.page_size];
                            r = p % a.c.page_size;
                        }
                        if (page >= 0 && page < a.c.num_pages)
                            box = (page * a.Hkv + h) * a.c.page_size + r;
                    }
                    boxes = __all_sync(kFull, lane >= nbox || box >= 0);
                }
                uint32_t valid = 0xf;
                if (!boxes) {
                    valid = 0;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int j = 4 * lane + u;
                        int p = -1;
                        if (tree) {
                            p = j < walk.w.nt ? walk.w.ctx + j : -1;
                        } else if (a.idx) {
                            if (base + j < a.top_k) {
                                p = a.idx[((size_t)b * a.Hkv + h) * a.top_k + base + j];
                                if (p < -1 || p >= walk.w.ctx) {
                                    flags |= kFlagIndexOutOfRange;
                                    p = -1;
                                }
                            }
                        } else {
                            p = base + j < walk.w.ctx ? base + j : -1;
                        }
                        rows[u] = a.oob_row;
                        if (p >= 0) {
                            int page = b, r = p;
                            if (a.c.table) {
                                page = a.c.table[(size_t)b * a.c.max_blocks + p / a.c.page_size];
                                r = p % a.c.page_size;
                            }
                            if (page >= 0 && page < a.c.num_pages) {
                                rows[u] = (page * a.Hkv + h) * a.c.page_size + r;
                                valid |= 1u << u;
                            } else {
                                flags |= kFlagPageOutOfRange;
                            }
                        }
                    }
                    if (flags)
                        atomicOr(a.status, flags);
                }
                const uint32_t word = __reduce_or_sync(0xffu << (lane & 24), valid << (4 * (lane & 7)));
                for (int kv = 0; ok && kv < 2; ++kv, ++e) {
                    const uint32_t slot = e % C::kSlots, use = e / C::kSlots;
                    if (use > 0)
                        ok = bar_wait(&bar_empty[slot], (use - 1) & 1, gave_up);
                    ok = __all_sync(kFull, ok);
                    if (!ok)
                        break;
                    if (kv == 0 && (lane & 7) == 0)
                        sm_valid[tile_no % kMaskRing][lane >> 3] = word;
                    __syncwarp();
                    if (lane == 0)
                        bar_expect(&bar_full[slot], kTileBytes);
                    __syncwarp();
                    const uint32_t dst = sm_ring + slot * kTileBytes;
                    if (boxes) {
                        if (box >= 0) {
                            const TmaDesc *map = kv ? &a.box_v : &a.box_k;
                            const uint32_t d = dst + lane * a.box_rows * 128;
                            tma_box(d, map, 0, box, &bar_full[slot]);
                            tma_box(d + kHalfBytes, map, 64, box, &bar_full[slot]);
                        }
                    } else {
                        const TmaDesc *map = kv ? &a.row_v : &a.row_k;
                        const uint32_t d = dst + lane * 4 * 128;
                        tma_rows4(d, map, 0, rows, &bar_full[slot]);
                        tma_rows4(d + kHalfBytes, map, 64, rows, &bar_full[slot]);
                    }
                }
            }
            walk.next(n);
        }
        if (!ok) {
            // leave no copy in flight: the last ones issued, each with a limit of its own
            int own_limit = 0;
            for (uint32_t k = e > C::kSlots ? e - C::kSlots : 0; k < e; ++k)
                bar_wait(&bar_full[k % C::kSlots], (k / C::kSlots) & 1, &own_limit);
        }
    } else if (warp == C::kSoftWarps + 1) {
        // ---- MMA issue.  One row tile: S of tile i + 1 is issued before P V of
        // tile i, so the tensor cores work while the softmax does.  Two row
        // tiles: they take turns.
        uint32_t e = 0;                  // ring entries consumed: 2 * tile (K), 2 * tile + 1 (V)
        uint32_t done_p[2] = {0, 0};     // P V issued per row tile (two row tiles)
        uint32_t segs[MT] = {};          // segments begun per row tile
        bool ok = true;
        auto issue_s = [&](uint32_t entry, int m, int buf, bool last) {
            if (lane == 0) {
                const uint32_t k = sm_ring + entry % C::kSlots * kTileBytes, q = sm_q + m * kTileBytes;
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t o = (s >> 2) * kHalfBytes + (s & 3) * 32;
                    mma_ss(tmem + buf * kTile, operand(q + o, 16), operand(k + o, 16), s > 0);
                }
                mma_commit(&bar_s[buf]);
                if (last)
                    mma_commit(&bar_empty[entry % C::kSlots]);
            }
            __syncwarp();
        };
        auto issue_o = [&](uint32_t entry, int m, int buf, bool first, bool last) {
            if (lane == 0) {
                const uint32_t v = sm_ring + entry % C::kSlots * kTileBytes;
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_ts(tmem + kColO + m * kTile, tmem + buf * kTile + s * 8,
                           operand(v + s * 16 * 128, kHalfBytes), !(first && s == 0));
                mma_commit(&bar_o[m]);
                if (last)
                    mma_commit(&bar_empty[entry % C::kSlots]);
            }
            __syncwarp();
        };
        auto wait_full = [&](uint32_t entry) {
            ok = ok && bar_wait(&bar_full[entry % C::kSlots], (entry / C::kSlots) & 1, gave_up);
            ok = __all_sync(kFull, ok);
            tmem_after();
        };
        auto wait_bar = [&](uint64_t *bar, uint32_t phase) {
            ok = ok && bar_wait(bar, phase & 1, gave_up);
            ok = __all_sync(kFull, ok);
            tmem_after();
        };
        while (ok && walk.left > 0) {
            const int n = walk.count();
            const int nm = MT == 1 ? 1 : (walk.rows() + kTile - 1) / kTile;
            for (int m = 0; m < nm; ++m)
                wait_bar(&bar_q[m], segs[m]++);
            if (!ok)
                break;
            if constexpr (MT == 1) {
                // tile i uses S buffer (global tile number) & 1
                const uint32_t g0 = e >> 1;
                wait_full(e);
                if (ok)
                    issue_s(e, 0, g0 & 1, true);
                for (int i = 0; ok && i < n; ++i) {
                    const uint32_t g = g0 + i;
                    if (i + 1 < n) {
                        wait_full(2 * (g + 1));
                        if (!ok)
                            break;
                        issue_s(2 * (g + 1), 0, (g + 1) & 1, true);
                    }
                    wait_bar(&bar_p[g & 1], g >> 1);
                    wait_full(2 * g + 1);
                    if (!ok)
                        break;
                    issue_o(2 * g + 1, 0, g & 1, i == 0, true);
                }
                e += 2 * n;
            } else {
                wait_full(e);
                if (ok)
                    for (int m = 0; m < nm; ++m)
                        issue_s(e, m, m, m == nm - 1);
                for (int i = 0; ok && i < n; ++i, e += 2) {
                    for (int m = 0; ok && m < nm; ++m) {
                        wait_bar(&bar_p[m], done_p[m]);
                        if (m == 0)
                            wait_full(e + 1);
                        if (!ok)
                            break;
                        ++done_p[m];
                        issue_o(e + 1, m, m, i == 0, m == nm - 1);
                        if (i + 1 < n) {
                            if (m == 0)
                                wait_full(e + 2);
                            if (!ok)
                                break;
                            issue_s(e + 2, m, m, m == nm - 1);
                        }
                    }
                }
            }
            walk.next(n);
        }
        if (!ok) {
            int own_limit = 0;
            if (lane == 0)
                mma_commit(&bar_drain);
            __syncwarp();
            bar_wait(&bar_drain, 0, &own_limit);
        }
    } else {
        // ---- softmax: thread r of a row tile owns query row r
        const int m = MT == 1 ? 0 : warp >> 2;
        const int r = (warp & 3) * 32 + lane;                 // row of the row tile, TMEM lane
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;    // this warp's TMEM lanes
        const float sl2 = a.scale * kLog2e;
        uint32_t count = 0;                                   // tiles done
        uint32_t tile_no = 0;                                 // tiles of the CTA before the segment
        uint32_t scans = 0;                                   // clearings of V with two row tiles
        bool ok = true;
        while (ok && walk.left > 0) {
            const int n = walk.count();
            const int unit_rows = walk.rows();
            const int nm = MT == 1 ? 1 : (unit_rows + kTile - 1) / kTile;
            if (m >= nm) {
                tile_no += n;
                walk.next(n);
                continue;
            }
            const int b = walk.b, h = walk.h;
            const int row0 = walk.m * MT * kTile + m * kTile;   // first query row of the row tile
            const int total_rows = walk.w.nt * a.G;
            const size_t q0 = (size_t)b * a.T * a.Hq + h * a.G;
            // Q row tile: chunk c of row x at x * 128 + ((c ^ x) & 7) * 16 of its half
            {
                const int x0 = (warp & 3) * 32;
#pragma unroll 4
                for (int it = 0; it < 16; ++it) {
                    const int x = x0 + it * 2 + (lane >> 4), c = lane & 15;
                    const int row = row0 + x;
                    uint4 val = make_uint4(0u, 0u, 0u, 0u);
                    if (row < total_rows)
                        val = *reinterpret_cast<const uint4 *>(
                            a.q + (q0 + (size_t)(row / a.G) * a.Hq + row % a.G) * kHeadDim + c * 8);
                    const uint32_t dst = sm_q + m * kTileBytes + (c >> 3) * kHalfBytes + x * 128 +
                                         (((c ^ x) & 7) << 4);
                    sts4(dst, val.x, val.y, val.z, val.w);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&bar_q[m]);
            }
            const int row = row0 + r;
            const int tok = row / a.G;                         // drafted token of this row
            const bool live = row < total_rows;
            const bool warp_live = row0 + (warp & 3) * 32 < total_rows;
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
            for (int i = 0; ok && i < n; ++i, ++count) {
                const int buf = MT == 1 ? (int)(count & 1) : m;
                const uint32_t phase = MT == 1 ? count >> 1 : count;
                const bool tree = walk.t + i == walk.w.tiles - 1;
                ok = __all_sync(kFull, bar_wait(&bar_s[buf], phase & 1, gave_up));
                if (!ok)
                    break;
                tmem_after();
                if (tree) {
                    // A V value that is not finite must not meet the zero
                    // probabilities of rows that do not see its token: such values
                    // leave the tile here and join the rows that do see it below.
                    // With two row tiles both look, then the first one clears.
                    const uint32_t entry = 2 * (tile_no + i) + 1;
                    ok = __all_sync(kFull, bar_wait(&bar_full[entry % C::kSlots],
                                                    (entry / C::kSlots) & 1, gave_up));
                    if (!ok)
                        break;
                    const uint32_t v = sm_ring + entry % C::kSlots * kTileBytes + r * 128;
                    bool any = false;
                    if (r < walk.w.nt) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            uint32_t x[4];
                            lds4(v + (c >> 3) * kHalfBytes + (((c ^ r) & 7) << 4), x);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                any |= (x[k] & 0x7f80u) == 0x7f80u || (x[k] & 0x7f800000u) == 0x7f800000u;
                        }
                    }
                    const uint32_t bits = __ballot_sync(kFull, any);
                    if (lane == 0)
                        sm_badv[m][warp & 3] = bits;
                    if constexpr (MT > 1) {
                        if (nm > 1 && m == 1 && lane == 0)
                            bar_arrive(&bar_scan);
                        if (nm > 1 && m == 0) {
                            ok = __all_sync(kFull, bar_wait(&bar_scan, scans & 1, gave_up));
                            if (!ok)
                                break;
                            ++scans;
                        }
                    }
                    if (m == 0 && bits) {
                        if (any) {
                            for (int c = 0; c < 16; ++c) {
                                uint32_t x[4];
                                const uint32_t at = v + (c >> 3) * kHalfBytes + (((c ^ r) & 7) << 4);
                                lds4(at, x);
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
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                    }
                }
                if (warp_live) {
                    const uint32_t at = tmem + buf * kTile + lanes;
                    uint32_t w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        w[c] = sm_valid[(tile_no + i) % kMaskRing][c];
                        if (tree)
                            w[c] &= sees[c];
                    }
                    const bool masked = (w[0] & w[1] & w[2] & w[3]) != 0xffffffffu;
                    // One row tile: the row's 128 scores stay in registers.  Two
                    // row tiles (12 warps' worth of registers): 32 at a time, read
                    // from tensor memory once for the maximum and once for the
                    // exponentials.
                    constexpr int kHeld = MT == 1 ? kTile : 32;
                    float s[kHeld];
                    auto fetch = [&](int c) {     // scores 32c .. 32c + 31 to s
                        float *d = s + (MT == 1 ? 32 * c : 0);
                        tmem_ld32(at + 32 * c, reinterpret_cast<uint32_t *>(d));
                    };
                    auto hide = [&](int c) {
                        float *d = s + (MT == 1 ? 32 * c : 0);
                        if (masked) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!(w[c] >> k & 1u))
                                    d[k] = -CUDART_INF_F;
                        }
                    };
                    float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                    __syncwarp();
                    if constexpr (MT == 1) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            fetch(c);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            tmem_loaded(reinterpret_cast<uint32_t *>(s) + 32 * c);
                    }
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if constexpr (MT > 1) {
                            fetch(c);
                            tmem_wait_ld();
                            tmem_loaded(reinterpret_cast<uint32_t *>(s));
                        }
                        hide(c);
                        const float *d = s + (MT == 1 ? 32 * c : 0);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            mx[k & 3] = fmaxf(mx[k & 3], d[k]);
                    }
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                    if (mref == -CUDART_INF_F)
                        mref = top;          // nothing summed so far: l = 0 and O = 0
                    // The running maximum lags until a row exceeds it by 2^8: the
                    // probabilities stay below 2^8 and the rescaling of O is rare.
                    const bool grow = i > 0 && top > mref + 8.0f;
                    if (__any_sync(kFull, grow)) {
                        ok = __all_sync(kFull, bar_wait(&bar_o[m], (count - 1) & 1, gave_up));
                        if (!ok)
                            break;
                        tmem_after();
                        const float mn = grow ? top : mref;
                        const float f = grow ? ex2(mref - mn) : 1.0f;
                        mref = mn;
                        l *= f;
                        const uint32_t o = tmem + kColO + m * kTile + lanes;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t x[32];
                            tmem_ld32(o + 32 * c, x);
                            tmem_wait_ld();
                            tmem_loaded(x);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
                            tmem_st32(o + 32 * c, x);
                        }
                    }
                    const float off = mref == -CUDART_INF_F ? 0.0f : -mref;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if constexpr (MT > 1) {
                            fetch(c);
                            tmem_wait_ld();
                            tmem_loaded(reinterpret_cast<uint32_t *>(s));
                            hide(c);
                        }
                        const float *d = s + (MT == 1 ? 32 * c : 0);
                        uint32_t p[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float p0 = ex2(fmaf(d[2 * k], sl2, off));
                            const float p1 = ex2(fmaf(d[2 * k + 1], sl2, off));
                            sum[(2 * k) & 3] += p0;
                            sum[(2 * k + 1) & 3] += p1;
                            p[k] = pack_bf16(p0, p1);
                        }
                        tmem_st16(at + 16 * c, p);   // over scores that have been read
                    }
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    tmem_wait_st();
                }
                tmem_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&bar_p[buf]);
            }
            if (!ok)
                break;
            // ---- the segment's result
            ok = __all_sync(kFull, bar_wait(&bar_o[m], (count - 1) & 1, gave_up));
            if (!ok)
                break;
            tmem_after();
            if (warp_live) {
                const bool whole = n == walk.w.tiles;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const int part = 2 * blockIdx.x + (walk.first ? 0 : 1);
                const size_t prow = (size_t)part * a.part_rows + m * kTile + r;
                uint32_t bad[4] = {0, 0, 0, 0};
                if (has_tree)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        bad[w] = sm_badv[m][w] & sees[w];
                const uint32_t o = tmem + kColO + m * kTile + lanes;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t x[32];
                    tmem_ld32(o + 32 * c, x);
                    tmem_wait_ld();
                    tmem_loaded(x);
                    if (live && (bad[0] | bad[1] | bad[2] | bad[3])) {
                        for (int j = 0; j < walk.w.nt; ++j) {
                            if (!(bad[j >> 5] >> (j & 31) & 1u))
                                continue;
                            const int p = walk.w.ctx + j;
                            int page = b, rr = p;
                            if (a.c.table) {
                                page = a.c.table[(size_t)b * a.c.max_blocks + p / a.c.page_size];
                                rr = p % a.c.page_size;
                            }
                            if (page < 0 || page >= a.c.num_pages)
                                continue;
                            const uint16_t *v =
                                a.c.v + (((size_t)page * a.Hkv + h) * a.c.page_size + rr) * kHeadDim + 32 * c;
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if ((v[k] & 0x7f80) == 0x7f80)
                                    x[k] = __float_as_uint(__uint_as_float(x[k]) +
                                                           __uint_as_float((uint32_t)v[k] << 16));
                        }
                    }
                    if (live && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            a.out + (q0 + (size_t)tok * a.Hq + row % a.G) * kHeadDim + 32 * c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint4 y;
                            y.x = pack_bf16(__uint_as_float(x[8 * k]) * inv, __uint_as_float(x[8 * k + 1]) * inv);
                            y.y = pack_bf16(__uint_as_float(x[8 * k + 2]) * inv, __uint_as_float(x[8 * k + 3]) * inv);
                            y.z = pack_bf16(__uint_as_float(x[8 * k + 4]) * inv, __uint_as_float(x[8 * k + 5]) * inv);
                            y.w = pack_bf16(__uint_as_float(x[8 * k + 6]) * inv, __uint_as_float(x[8 * k + 7]) * inv);
                            dst[k] = y;
                        }
                    } else if (live) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.part_o + prow * kHeadDim + 32 * c);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            dst[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                    }
                    __syncwarp();
                }
                if (!whole && live) {
                    a.part_m[prow] = mref;
                    a.part_l[prow] = l;
                }
                tmem_before();
            }
            __syncwarp();
            tile_no += n;
            walk.next(n);
        }
    }
    tmem_before();
    __syncthreads();
    if (tid == 0 && sm_gave_up)
        atomicOr(a.status, kFlagWaitTimeout);
    if (warp == C::kSoftWarps + 1) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
    }
}

// Joins the parts of the units that several CTAs shared.  CTA x is given the
// unit, if any, whose first cut is the end of range x; its warps take the
// unit's rows in turn: o = sum_s o_s 2^(m_s - m) / sum_s l_s 2^(m_s - m).
constexpr int kJoinWarps = 4;

template <int MT>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ TreeArgs a,
                                                                     int ctas)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long total = a.prefix[a.B];
    const long long per = (total + ctas - 1) / ctas;
    const int c = blockIdx.x + 1;
    const long long pos = c * per;
    if (pos >= total)
        return;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.prefix[mid] <= pos)
            lo = mid;
        else
            hi = mid - 1;
    }
    uint32_t bad = 0;
    const Work w = work_of<MT>(a, lo, bad);
    const long long unit = (pos - a.prefix[lo]) / w.tiles;
    const long long u0 = a.prefix[lo] + unit * w.tiles;
    if (u0 == pos || u0 / per != c - 1)
        return;
    const int c0 = c - 1, c1 = (int)((u0 + w.tiles - 1) / per);
    const int h = (int)(unit / w.blocks), m = (int)(unit % w.blocks);
    const int rows = min(w.nt * a.G - m * MT * kTile, MT * kTile);
    auto part_row = [&](int cc, int r) {
        const int part = 2 * cc + (u0 > cc * per ? 1 : 0);
        return (size_t)part * a.part_rows + r;
    };
    for (int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r < rows; r += gridDim.y * kJoinWarps) {
        float top = -CUDART_INF_F;
        for (int cc = c0 + lane; cc <= c1; cc += 32)
            top = fmaxf(top, a.part_m[part_row(cc, r)]);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        float l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int cc = c0; cc <= c1; ++cc) {
            const size_t p = part_row(cc, r);
            const float ms = a.part_m[p];
            const float4 x = *reinterpret_cast<const float4 *>(a.part_o + p * kHeadDim + lane * 4);
            const float f = ms == -CUDART_INF_F ? 0.0f : exp2f(ms - top);
            if (f != 0.0f) {      // an empty part has nothing to add
                l += a.part_l[p] * f;
                o.x += x.x * f;
                o.y += x.y * f;
                o.z += x.z * f;
                o.w += x.w * f;
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int row = m * MT * kTile + r;
        uint2 y;
        y.x = pack_bf16(o.x * inv, o.y * inv);
        y.y = pack_bf16(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2 *>(
            a.out + (((size_t)lo * a.T + row / a.G) * a.Hq + h * a.G + row % a.G) * kHeadDim + lane * 4) = y;
    }
}

template <int MT>
cudaError_t launch(const TreeArgs &a, int sms, cudaStream_t stream)
{
    using C = Cfg<MT>;
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !ready[dev]) {
            err = cudaFuncSetAttribute(tree_attention_kernel<MT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
            if (err != cudaSuccess)
                return err;
            if (dev >= 0 && dev < 64)
                ready[dev] = true;
        }
    }
    const int ctas = sms < kMaxTreeCtas ? sms : kMaxTreeCtas;
    tree_attention_kernel<MT><<<ctas, C::kThreads, C::kSmem, stream>>>(a);
    err = cudaGetLastError();
    if (err != cudaSuccess || ctas < 2)
        return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas - 1, (a.part_rows + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_join_kernel<MT>, a, ctas);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeArgs &a, int sms, cudaStream_t stream)
{
    return a.T * a.G <= kTile ? launch<1>(a, sms, stream) : launch<2>(a, sms, stream);
}

}  // namespace td
