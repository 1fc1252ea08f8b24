// td_prompt.cu -- attention of a packed batch of new tokens (prompts, chunks of prompts,
// single tokens) over a cache of 16- or 4-bit rows: causal, with a sliding window and a
// few first tokens that stay visible, or without.
//
// New token i of request b stands at position p = seq_lens[b] - n_b + i; query head h,
// KV head g = h / G:
//     S = { j <= p : j < sinks or p - j < window }    (window 0: every j <= p),
//     out = sum_{j in S} softmax(scale q . K_j) V_j   (0 for empty S)
// by an online softmax over tiles of 128 cached tokens.
//
// A unit of work is 256 query rows (tokens x the G heads) of one request and KV head, as two
// row tiles of 128.  S = Q K^T and O += P V run on the tensor cores (tcgen05.mma; Q, K, V
// in shared memory, S, P, O in tensor memory); while one row tile's softmax runs, the tensor
// cores have the other's products.  K and V tiles serve both row tiles and are copied row
// by row, so any page size and any window edge is alike.  4-bit rows are decoded to fp16 on
// their way into shared memory, where they are exact; q and P are then fp16 too (q times
// a power of two per row).
//
// Measured on GB300 (a call in a graph; rates of the visible products alone):
//   5 prompts of 1021 .. 6144 tokens, 32 query / 8 KV heads, window 1024: 181 us, 1.10 PFLOP/s
//   3 chunks of 517 .. 1024 tokens on 5K .. 16K tokens in 4 bits:          393 us, 1.17 PFLOP/s
// A step of 64 tokens is 1272 cycles of MMAs (S with N = 64 reads its Q from shared memory as often
// as with 128: 380 cycles a row tile, not 256) and about as many of shared memory's, and takes
// 1700: the softmax warps and the copies share the issue slots (55% taken) and wait on one another.
// Tried and slower: S of 128 tokens (the row tiles' products fall into step: 4800 cycles where two steps
// take 3900), S in two places with P over it (205 us), two threads per row (216 and 487 us), results
// read out behind the next unit's first step (209 and 420), rows stored 32 bytes a lane (186 and 398).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "td_attn_common.cuh"
#include "td_cache.h"
#include "td_tc.cuh"

namespace td {
namespace {

constexpr int kTile = 128;                       // tokens per tile, query rows per row tile
constexpr int kHalfBytes = kTile * 128;          // one 64-value half of a tile's rows
constexpr int kTileBytes = 2 * kHalfBytes;
constexpr int kUnitRows = kPromptRows;
static_assert(kUnitRows == 2 * kTile, "two row tiles");
// A unit's begin and end cost as much as two tiles: it counts as so many more.  (Prompts of 1K-6K,
// window 1024, ranges cut by tiles alone: 230 us with 10 units per CTA, 344 with 46.)
constexpr int kUnitCost = 2;
// A range's begin within so much of a unit's begin or end moves there: what a cut costs (another
// begin and end, the join) is more than the SMs would differ by.  Units of up to twice that are whole.
// In units of kLong ranges and more only within kSnapLong: they are cut all the same, and there a range
// that is moved leaves SMs idle.  (2 requests of 2000 tokens, 100 of them new: 29.6 -> 24.7 us, over 4-bit
// rows 46.4 -> 35.1; kSnapLong for every unit: mixed steps 27 -> 35 us, prompts 181 -> 189.)
constexpr int kSnap = 6, kSnapLong = 2, kLong = 3;
static_assert(kSnap >= kUnitCost && kSnapLong >= kUnitCost, "every part of a unit has a tile");
constexpr int kLeastCost = 4;                    // of a CTA's range
constexpr int kMostSlots = 5;
// Ring of K and V tiles: 16-bit rows 5; 4-bit rows 4, and rings of the copy warps' coded rows.
template <bool Q4> constexpr int kRingSlots = Q4 ? 4 : 5;
constexpr int kRawRing = 3;                      // K or V rows of a copy warp on their way
constexpr int kRawBytes = 32 * (kCodeBytes + 8);
constexpr int kMaskRing = 8;
constexpr int kSoftWarps = 8;                    // four per row tile
constexpr int kCopier = 8, kCopiers = 4;         // copy warps
constexpr int kSched = 12, kIssuer = 13, kIssuers = 2;      // an issuer per row tile
constexpr int kThreads = 32 * 15;
constexpr int kStep = 64;                        // tokens of one S
constexpr int kCopyRows = kTile / kCopiers;      // of a tile, per copy warp: one a lane
static_assert(kCopyRows == 32, "a lane has one row of a tile");
constexpr int kUnitRing = 4;
constexpr float kMostSum = 8192.0f;              // of a step's P of a row (fp16 ends at 65504)
constexpr float kMostFloat = 3.402823466e38f;
constexpr int kUnitUsers = kSoftWarps + kCopiers + kIssuers;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;      // O of row tile t: kColO + 128 t; S: 128 t
constexpr uint32_t kColP = 64;       // two P of a row tile: behind its S, 32 columns each
constexpr size_t kSmem = (size_t)(2 + kMostSlots) * kTileBytes + 3 * 1024;    // + Extra

// A unit of work, as every role reads it.
struct Unit {
    int b, h;
    int q0;            // first row of q of the request
    int row0, rows;    // query rows of the request: row = token * G + head
    int pos0;          // position of the request's first new token
    // The tokens that some row may see, one behind the other: the first ones (positions 0 ..
    // first - 1), then positions low .. low + rest - 1.  Tiles are cut from this list.
    int first, low, rest;
    // The CTA's segment: tiles of 128 tokens from tile0 on, steps of 64; tiles -1: no more.
    int tile0, tiles, steps;
    int part;          // where its result goes: partial sums number `part`, -1: it is the unit's whole
};

// Where a CTA's range of tiles begins.
struct Start {
    int b, block, h, at;     // request, block of query rows, KV head, cost of the unit that lies before
    long long begin, end;    // of the range, in the batch's cost
};

// Who arrives and who waits; a wait looks at a phase's parity, so each must come when
// the phase before is over and before the one after can be.  Step number g of a row tile, over
// units: its P has buffer g & 1.
//   full     a ring slot's use: 16-bit rows: every copy thread as its copies land (then fenced by
//            the issuers), and each copy warp behind its word of `valid`; 4-bit rows: each copy
//            warp when its rows are written and fenced.  Both issuers wait for every one in order.
//   empty    each issuer's commit behind its MMAs that read the slot, or, in a unit without its row
//            tile, its arrival behind `full`; the copy warps wait for every use.
//   q, q_free   as full and empty, per unit.
//   s[t]     S of step g of row tile t.  Its softmax warps wait for every one.
//   r[t]     the row tile's 128 softmax threads have S of step g in registers.  Its issuer waits for
//            every one before it issues the S behind it.
//   p[t][g & 1]  P of step g, the row tile's softmax threads; its issuer waits for every one,
//            and P of g + 2 needs S of g + 2, which is issued behind P V of g.
//   o[t][g & 1]  P V of a step.  The softmax waits for that of g - 2 before it writes P of g over
//            that step's, so for every one, and that of g + 2 needs a later P.  For that of g - 1 it
//            waits to rescale O, and behind a unit's last step.
//   unit_there, unit_free   a unit's entry, written by the scheduler and read by all other roles, who free
//            it when they are done with the unit.
// q_inv of a unit lies where that of the unit but one before did: its Q comes after q_free of the
// unit before, to which an issuer arrives behind all of the unit but one before, for which P was
// needed.
struct Extra {
    uint64_t full[kMostSlots], empty[kMostSlots];
    uint64_t q, q_free;
    uint64_t s[2], r[2], p[2][2], o[2][2];
    uint64_t unit_there[kUnitRing], unit_free[kUnitRing];
    uint64_t drain[kIssuers], done[kIssuers], never;
    Unit unit[kUnitRing];
    Start start;
    long long sums[kThreads / 32];
    alignas(16) uint32_t valid[kMaskRing][4];    // tokens of a tile that exist
    float q_inv[2][kUnitRows];                   // 4-bit rows: what a row's scores are multiplied by
    uint32_t tmem;
    Progress progress;
    Progress last_waits[kThreads / 32];
};
static_assert((2 + kMostSlots) * kTileBytes + sizeof(Extra) <= kSmem, "shared memory");
static_assert(kCopiers * kRawRing * kRawBytes <= kTileBytes, "coded rows take the fifth slot's place");

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Eight 4-bit values (one word of codes) times their scale, as fp16 pairs.
__device__ __forceinline__ void decode8(uint32_t codes, uint32_t scale, uint32_t (&x)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b32 w, x, y, z;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 w, a;\n\tcvt.rn.f16x2.e2m1x2 x, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 y, c;\n\tcvt.rn.f16x2.e2m1x2 z, d;\n\t"
        "mul.rn.f16x2 %0, w, %5;\n\tmul.rn.f16x2 %1, x, %5;\n\t"
        "mul.rn.f16x2 %2, y, %5;\n\tmul.rn.f16x2 %3, z, %5;\n\t}"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(codes), "r"(scale));
}

// The lowest n of 32 bits (n < 0: none, n > 32: all).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    uint32_t r;
    asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(r) : "r"(max(n, 0)));
    return r;
}

// Four neighbouring lanes' rows of two times four 16-byte pieces, turned: lane c of the four then
// has piece c of row k of the first four in y[4 k ..], of the others in y[16 + 4 k ..].
__device__ __forceinline__ void turn4(uint32_t (&y)[32], int lane)
{
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        const bool up = lane & d;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            if (p & d)
                continue;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t &lo = y[4 * p + k], &hi = y[4 * (p + d) + k];
                const uint32_t got = __shfl_xor_sync(kFull, up ? lo : hi, d);
                lo = up ? got : lo;
                hi = up ? hi : got;
            }
        }
    }
}

// Four consecutive values of a cached row, as they are held: two words of 16-bit values, or four codes and
// their scale.
template <bool Q4> __device__ __forceinline__ uint2 row_words(const RowsArgs &c, bool v, int row, int lane)
{
    const uint8_t *x = v ? c.v : c.k;
    if constexpr (!Q4)
        return *reinterpret_cast<const uint2 *>(x + (size_t)(uint32_t)row * (kHeadDim * 2) + 8 * lane);
    return make_uint2(*reinterpret_cast<const uint16_t *>(x + (size_t)(uint32_t)row * kCodeBytes + 2 * lane),
                      c.scales[(size_t)(uint32_t)row * kScaleBytes + (v ? 8 : 0) + lane / 4]);
}

template <bool Q4> __device__ __forceinline__ float4 row_values(uint2 y)
{
    if constexpr (!Q4)
        return make_float4(bf_lo(y.x), bf_hi(y.x), bf_lo(y.y), bf_hi(y.y));
    uint32_t lo, hi;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .b16 t;\n\t.reg .b32 w, x, s;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 w, a;\n\tcvt.rn.f16x2.e2m1x2 x, b;\n\t"
        "cvt.u16.u32 t, %3;\n\tcvt.rn.f16x2.e4m3x2 s, t;\n\t"
        "mul.rn.f16x2 %0, w, s;\n\tmul.rn.f16x2 %1, x, s;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(y.x), "r"(y.y | y.y << 8));
    const float2 f0 = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 f1 = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return make_float4(f0.x, f0.y, f1.x, f1.y);
}

// One query row by a warp, kWalk positions at a time: for rows whose tiles held values that are
// not finite, which in a product meet the zero probabilities of tokens that the row does not
// see.  Rare, and out of line: 16 prompts of 2000 tokens that all see a NaN in some dims take 266 ms, over
// 4-bit rows 243 (one position at a time 751 and 1124, eight 218 and 169, but then the kernel takes 395 us
// without a NaN where it takes 392), in all dims 3.4; without one 0.45 and 0.8.  `walked` (or
// null) counts on: a CTA's other roles wait for the warp, for longer than a wait without progress may take.
constexpr int kWalk = 4;

template <bool Q4>
__device__ __noinline__ void attend_row(const PromptArgs &a, int b, int h, int p, size_t q_row, int lane,
                                        uint32_t *walked)
{
    const uint2 y = *reinterpret_cast<const uint2 *>(a.q + q_row * kHeadDim + 4 * lane);
    const float4 q = make_float4(bf_lo(y.x), bf_hi(y.x), bf_lo(y.y), bf_hi(y.y));
    const Range w = window_range(p + 1, a.window, a.sinks);
    const int count = w.first + p + 1 - w.low;
    float m = -CUDART_INF_F, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int t0 = 0; t0 < count; t0 += kWalk) {
        if (walked && lane == 0)
            atomicAdd(walked, 1u);
        // lane k has the row of the k-th position (-1: none)
        const int t = t0 + lane % kWalk, j = t < w.first ? t : w.low + t - w.first;
        const int mine = t < count ? row_of(a.rows, a.Hkv, h, j, page_of(a.rows, b, j)) : -1;
        int rows[kWalk];
        uint2 kw[kWalk], vw[kWalk];
#pragma unroll
        for (int k = 0; k < kWalk; ++k)
            rows[k] = __shfl_sync(kFull, mine, k);
#pragma unroll
        for (int k = 0; k < kWalk; ++k) {
            kw[k] = row_words<Q4>(a.rows, false, max(rows[k], 0), lane);
            vw[k] = row_words<Q4>(a.rows, true, max(rows[k], 0), lane);
        }
        float x[kWalk], mn = m;
#pragma unroll
        for (int k = 0; k < kWalk; ++k) {
            const float4 key = row_values<Q4>(kw[k]);
            x[k] = fmaf(q.x, key.x, fmaf(q.y, key.y, fmaf(q.z, key.z, q.w * key.w)));
        }
#pragma unroll
        for (int d = 16; d; d >>= 1)
#pragma unroll
            for (int k = 0; k < kWalk; ++k)
                x[k] += __shfl_xor_sync(kFull, x[k], d);
#pragma unroll
        for (int k = 0; k < kWalk; ++k) {
            x[k] *= a.scale * kLog2e;
            mn = rows[k] >= 0 ? fmaxf(mn, x[k]) : mn;
        }
        // (a sum that is zero has nothing to keep, whatever the factor)
        const float f = safe_exp2_diff(m, mn), off = mn == -CUDART_INF_F ? 0.0f : mn;
        m = mn;
        l *= f;
        o.x *= f;
        o.y *= f;
        o.z *= f;
        o.w *= f;
#pragma unroll
        for (int k = 0; k < kWalk; ++k) {
            if (rows[k] < 0)
                continue;
            const float e = exp2f(x[k] - off);
            const float4 v = row_values<Q4>(vw[k]);
            l += e;
            o.x += e * v.x;
            o.y += e * v.y;
            o.z += e * v.z;
            o.w += e * v.w;
        }
        // (no later position makes a number of a NaN)
        const float all = fminf(fminf(fabsf(o.x), fabsf(o.y)), fminf(fabsf(o.z), fabsf(o.w)));   // (of the numbers)
        if (l != 0.0f && __all_sync(kFull, all != all))
            break;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 r;
    r.x = l == 0.0f ? 0u : pack_bf16(o.x * inv, o.y * inv);
    r.y = l == 0.0f ? 0u : pack_bf16(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2 *>(a.out + q_row * kHeadDim + 4 * lane) = r;
}

template <bool Q4>
__global__ void __launch_bounds__(kThreads, 1) prompt_attention_kernel(const __grid_constant__ PromptArgs a)
{
    constexpr int kSlots = kRingSlots<Q4>;
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    Extra &x = *reinterpret_cast<Extra *>(sm_raw + (2 + kMostSlots) * kTileBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sm_q = smem_of(sm_raw);
    const uint32_t sm_ring = sm_q + 2 * kTileBytes;
    volatile Progress *progress = &x.progress;
    auto bar_wait = [&](uint64_t *bar, unsigned parity) {
        return bar_wait_for(bar, parity & 1, progress, a.wait_cycles);
    };
    auto warp_wait = [&](uint64_t *bar, unsigned parity) {
        return (bool)__all_sync(kFull, bar_wait(bar, parity));
    };
    if (sm_q & 1023) {            // (cannot be: the swizzled tiles need it)
        pdl_wait();
        if (tid == 0) {
            atomicOr(a.status, kFlagWaitTimeout);
            a.ws->join[blockIdx.x] = PromptJoin{-1};
        }
        return;
    }
    if (tid == 32 * kIssuer) {
        x.progress = Progress{};
        for (int i = 0; i < kThreads / 32; ++i)
            x.last_waits[i] = Progress{};
        for (int i = 0; i < kSlots; ++i) {
            bar_init(&x.full[i], Q4 ? kCopiers : 33 * kCopiers);
            bar_init(&x.empty[i], kIssuers);
        }
        bar_init(&x.q, Q4 ? kCopiers : 32 * kCopiers);
        bar_init(&x.q_free, kIssuers);
        for (int t = 0; t < 2; ++t) {
            bar_init(&x.s[t], 1);
            bar_init(&x.r[t], kTile);
            for (int i = 0; i < 2; ++i) {
                bar_init(&x.p[t][i], kTile);
                bar_init(&x.o[t][i], 1);
            }
        }
        for (int i = 0; i < kUnitRing; ++i) {
            bar_init(&x.unit_there[i], 1);
            bar_init(&x.unit_free[i], kUnitUsers);
        }
        for (int t = 0; t < kIssuers; ++t) {
            bar_init(&x.drain[t], 1);
            bar_init(&x.done[t], 1);
        }
        bar_init(&x.never, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuer) {
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_of(&x.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_before();
    __syncthreads();
    tmem_after();
    // (all 512 columns are this CTA's, so they begin at 0)
    constexpr uint32_t tmem = 0;
    if (x.tmem != 0 && tid == 0)             // (cannot be)
        x.progress.gave_up = 1;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    // The next unit of a role: waits for its entry.  (n: units that the role has had.)
    uint32_t units = 0;
    bool ok = true;
    auto unit_entry = [&]() -> const Unit & { return x.unit[units % kUnitRing]; };
    auto next_unit = [&]() {
        ok = ok && warp_wait(&x.unit_there[units % kUnitRing], units / kUnitRing);
        return ok && unit_entry().tiles >= 0;
    };
    auto free_unit = [&]() {      // by one lane of a warp that is done with the unit
        bar_arrive(&x.unit_free[units % kUnitRing]);
    };

    // ---- the CTA's range: an equal, contiguous run of the batch's tiles, over units' borders, so that
    // no long context and no small batch leaves SMs idle; a unit that several CTAs share is
    // joined by prompt_join_kernel.  Units in order: request, block of 256 query rows, KV head.
    // Request b's blocks are numbers floor(cu[b] G / 256) + b and on (room for all of them; a number
    // without a block has no tiles).
    auto start_of = [&](int b) { return min(max(a.cu_new[b], 0), a.num_tokens); };
    auto number_of = [&](int b) { return (int64_t)start_of(b) * a.G / kUnitRows + b; };
    uint32_t bad = 0;
    struct Request {
        int b, q0, count, n, blocks;
    };
    auto request = [&](int b) {
        Request r;
        r.b = b;
        r.q0 = start_of(b);
        r.count = max(0, start_of(b + 1) - r.q0);
        r.blocks = (int)(((int64_t)r.count * a.G + kUnitRows - 1) / kUnitRows);
        r.n = seq_len_of(a.seq_lens, b, a.Nmax, bad);
        if (r.count > r.n)
            bad |= kFlagSeqLenOutOfRange;
        return r;
    };
    auto unit_of = [&](const Request &r, int block, int h) {
        Unit u;
        u.b = r.b;
        u.h = h;
        u.q0 = r.q0;
        u.row0 = block * kUnitRows;
        u.rows = min(r.count * a.G - u.row0, kUnitRows);
        u.pos0 = r.n - r.count;                   // (below zero: those tokens see nothing)
        const int p0 = u.pos0 + (u.row0 >> a.g_shift);
        const int p1 = u.pos0 + ((u.row0 + u.rows - 1) >> a.g_shift);
        u.low = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
        u.first = min(a.sinks, u.low);
        u.rest = max(p1 + 1 - u.low, 0);
        u.tile0 = 0;
        u.steps = max(1, (u.first + u.rest + kStep - 1) / kStep);
        u.tiles = (u.steps + 1) / 2;
        u.part = -1;
        return u;
    };
    int64_t per;
    auto snap_of = [&](int cost) { return cost >= kLong * per ? kSnapLong : kSnap; };
    {
        const int64_t numbers = (int64_t)a.num_tokens * a.G / kUnitRows + a.B;
        const int64_t run = (numbers + kThreads - 1) / kThreads;
        const int64_t n0 = min(tid * run, numbers), n1 = min(n0 + run, numbers);
        int b0 = 0;                               // the last request that begins at or before number n0
        for (int hi = a.B; hi - b0 > 1;) {
            const int mid = (b0 + hi) >> 1;
            if (number_of(mid) <= n0)
                b0 = mid;
            else
                hi = mid;
        }
        // Calls f(request, block, tiles) for the run's blocks, until it returns false.
        auto walk = [&](auto f) {
            if (n0 >= n1)
                return;
            int b = b0;
            Request r = request(b);
            int64_t first = number_of(b), next = number_of(b + 1);
#pragma unroll 1
            for (int64_t n = n0; n < n1; ++n) {
                while (b + 1 < a.B && n >= next) {
                    r = request(++b);
                    first = next;
                    next = number_of(b + 1);
                }
                if (n - first >= 0 && n - first < r.blocks && !f(r, (int)(n - first), unit_of(r, (int)(n - first), 0).tiles))
                    return;
            }
        };
        long long mine = 0;
        walk([&](const Request &, int, int tiles) {
            mine += (long long)(tiles + kUnitCost) * a.Hkv;
            return true;
        });
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
            x.sums[warp] = inc;
        if (tid == 0)
            x.start.begin = x.start.end = 0;
        __syncthreads();
        long long all = 0, at0 = inc - mine;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp)
                at0 += x.sums[i];
            all += x.sums[i];
        }
        per = max((all + gridDim.x - 1) / gridDim.x, (long long)kLeastCost);
        // Where the range begins and ends: the unit there, the place in it, moved to its begin or end
        // where that is near.
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const long long target = (blockIdx.x + k) * per;
            long long at = at0;
            if (target < all && at <= target && target < at + mine)
                walk([&](const Request &r, int block, int tiles) {
                    const int cost = tiles + kUnitCost;
                    if (target >= at + (long long)cost * a.Hkv) {
                        at += (long long)cost * a.Hkv;
                        return true;
                    }
                    const int h = (int)(target - at) / cost, in = (int)(target - at) - h * cost;
                    const int snap = snap_of(cost), to = in <= snap ? 0 : cost - in <= snap ? cost : in;
                    if (k == 0) {
                        x.start.b = r.b;
                        x.start.block = block;
                        x.start.h = h;
                        x.start.at = to;
                        x.start.begin = target - in + to;
                    } else {
                        x.start.end = target - in + to;
                    }
                    return false;
                });
            else if (target >= all && tid == 0) {
                if (k == 0)
                    x.start.begin = all;
                else
                    x.start.end = all;
            }
        }
        __syncthreads();
    }
    // The unit behind a place's.  (False: there is none, which no cu_new that ascends leads to.)
    auto next_unit_of = [&](Start &w, Request &r) {
        w.at = 0;
        if (++w.h < a.Hkv)
            return true;
        w.h = 0;
        if (++w.block < r.blocks)
            return true;
        w.block = 0;
        do {
            if (r.b + 1 >= a.B)
                return false;
            r = request(r.b + 1);
        } while (r.blocks == 0);
        w.b = r.b;
        return true;
    };
    // Publishes the CTA's units (the scheduler, as far ahead as there are entries).
    auto publish_all = [&] {
        Start w = x.start;
        long long left = w.end - w.begin;
        Request r{};
        PromptJoin join{-1};
        if (left > 0) {
            r = request(w.b);
            const Unit u = unit_of(r, w.block, w.h);
            if (w.at == u.tiles + kUnitCost) {
                if (!next_unit_of(w, r))
                    left = 0;
                const Unit v = unit_of(r, w.block, w.h);
                join = PromptJoin{v.b, v.h, v.q0, v.row0, 0, v.pos0, 0};
            } else {
                // Is this the first cut of the unit?  The last CTA that has a part of it begins at
                // least snap + 1 before its end.
                const int snap = snap_of(u.tiles + kUnitCost);
                const bool cut = w.at > 0 && w.at - per <= snap;
                join = PromptJoin{u.b, u.h, u.q0, u.row0, cut ? u.rows : 0, u.pos0,
                                  (int)((w.begin - w.at + u.tiles + kUnitCost - snap - 1) / per)};
            }
        }
        if (lane == 0)
            a.ws->join[blockIdx.x] = join;
#pragma unroll 1
        for (uint32_t n = 0;; ++n) {
            Unit u;
            u.tiles = -1;
            if (left > 0) {
                // Of cost at .. end of the unit; its first kUnitCost are no tiles.
                u = unit_of(r, w.block, w.h);
                const int all = u.tiles;
                const int end = (int)min((long long)(all + kUnitCost), w.at + left);
                u.tile0 = max(w.at - kUnitCost, 0);
                u.tiles = end - kUnitCost - u.tile0;
                u.steps = min(u.steps - 2 * u.tile0, 2 * u.tiles);
                if (u.tiles < all)
                    u.part = 2 * blockIdx.x + (n > 0);
                left -= end - w.at;
                if (left > 0 && !next_unit_of(w, r))
                    left = 0;
            }
            if (n >= kUnitRing)
                ok = warp_wait(&x.unit_free[n % kUnitRing], n / kUnitRing - 1);
            if (ok && lane == 0) {
                x.unit[n % kUnitRing] = u;
                bar_arrive(&x.unit_there[n % kUnitRing]);
            }
            __syncwarp();
            if (!ok || u.tiles < 0)
                break;
        }
    };

    if (warp == kSched) {
        publish_all();
    } else if (warp >= kCopier && warp < kCopier + kCopiers) {
        // ---- copy warps: a unit's Q, then its K and V tiles, kCopyRows rows of each per warp
        const int me = warp - kCopier;
        uint32_t e = 0;                           // ring entries begun
        uint32_t flags = 0;
        uint32_t tile_no = 0;
        auto arrive = [&](uint64_t *bar) {        // this warp's rows are written: the MMAs may read them
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                bar_arrive(bar);
        };
#pragma unroll 1
        for (; next_unit(); ++units) {
            const Unit u = unit_entry();
            // The row of this lane's token of tile j, in three steps for later tiles while
            // earlier ones are copied: position, page, row.
            auto position = [&](int j) {
                const int t = (u.tile0 + j) * kTile + kCopyRows * me + lane;
                return j >= u.tiles || t >= u.first + u.rest ? -1 : t < u.first ? t : t - u.first + u.low;
            };
            auto page = [&](int p) { return p >= 0 ? page_of(a.rows, u.b, p) : 0; };
            auto find = [&](int p, int pg) {
                if (p < 0)
                    return -1;
                const int row = row_of(a.rows, a.Hkv, u.h, p, pg);
                if (row < 0)
                    flags |= kFlagPageOutOfRange;
                return row;
            };
            int p1 = position(0), p2 = position(1);
            int pg1 = page(p1), pg2 = page(p2);
            auto next_row = [&](int j) {          // of tile j, one after the other
                const int row = find(p1, pg1);
                p1 = p2, pg1 = pg2;
                p2 = position(j + 2), pg2 = page(p2);
                return row;
            };
            // Waits for the next ring slot; behind K's the tile's word of `valid`.
            auto next_slot = [&](bool k, uint32_t there) {
                const uint32_t slot = e % kSlots, use = e / kSlots;
                if (use > 0)
                    ok = ok && warp_wait(&x.empty[slot], use - 1);
                if (ok && k && lane == 0)
                    x.valid[tile_no % kMaskRing][me] = there;
                ++e;
                return slot;
            };
            // Q, half a warp per row of 256 bytes, behind the first K tile: its place is free only when
            // the last S of the unit before is done.
            auto copy_q = [&] {
                if (units > 0)
                    ok = warp_wait(&x.q_free, units - 1);
                if (!ok)
                    return;
                const int c = lane & 15;
                const uint16_t *src = a.q + ((size_t)u.q0 * a.Hq + (size_t)u.h * a.G) * kHeadDim + c * 8;
                const uint32_t dst = sm_q + (c >> 3) * kHalfBytes;
#pragma unroll 8
                for (int r = 2 * me + (lane >> 4); r < u.rows; r += 2 * kCopiers) {
                    const int row = u.row0 + r, tk = row >> a.g_shift, g = row & (a.G - 1);
                    const uint32_t to = dst + (r >> 7) * kTileBytes + (r & 127) * 128 + (((c ^ r) & 7) << 4);
                    const uint16_t *from = src + ((size_t)tk * a.Hq + g) * kHeadDim;
                    if constexpr (!Q4) {
                        copy16(to, from, true);
                    } else {
                        // times a power of two that brings the row's largest value to 2^8: values
                        // 2^-22 times as large keep all their bits in fp16
                        const uint4 y = *reinterpret_cast<const uint4 *>(from);
                        uint32_t w[4] = {y.x, y.y, y.z, y.w}, top = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            top = __vmaxu2(top, w[k] & 0x7fff7fffu);
                        top = max(top & 0xffffu, top >> 16);
                        const unsigned half = 0xffffu << (lane & 16);
#pragma unroll
                        for (int d = 8; d; d >>= 1)
                            top = max(top, __shfl_xor_sync(half, top, d));
                        const int ex = top >> 7;
                        const int up = ex == 0 || ex == 255 ? 0 : max(-120, min(120, 135 - ex));
                        const float f = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack_f16(bf_lo(w[k]) * f, bf_hi(w[k]) * f);
                        sts4(to, w[0], w[1], w[2], w[3]);
                        if (c == 0)
                            x.q_inv[units & 1][r] = __uint_as_float((uint32_t)(127 - up) << 23);
                    }
                }
                if constexpr (!Q4)
                    copies_arrive(&x.q);
                else
                    arrive(&x.q);
            };
            if constexpr (!Q4) {
#pragma unroll 1
                for (int j = 0; j < u.tiles && ok; ++j, ++tile_no) {
                    const int row = next_row(j);
                    const uint32_t there = __ballot_sync(kFull, row >= 0);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t slot = next_slot(kv == 0, there);
                        if (!ok)
                            break;
                        // half a warp per row of 256 bytes: rows 0 .. 15, and 16 .. 31
                        const int c = lane & 15;
                        const uint8_t *src = (kv ? a.rows.v : a.rows.k) + c * 16;
                        const uint32_t dst = sm_ring + slot * kTileBytes + (c >> 3) * kHalfBytes +
                                             (kCopyRows * me + (lane & 16)) * 128 + ((c & 7) << 4);
                        if (there == kFull) {
#pragma unroll
                            for (int r = 0; r < 16; ++r) {
                                const int from = __shfl_sync(kFull, row, r, 16);
                                copy16((dst ^ ((r & 7) << 4)) + r * 128, src + (size_t)(uint32_t)from * (kHeadDim * 2));
                            }
                        } else {
#pragma unroll 1
                            for (int r = 0; r < 16; ++r) {
                                const int from = __shfl_sync(kFull, row, r, 16);
                                copy16((dst ^ ((r & 7) << 4)) + r * 128,
                                       src + (size_t)(uint32_t)max(from, 0) * (kHeadDim * 2), from >= 0);
                            }
                        }
                        copies_arrive(&x.full[slot]);
                        if (lane == 0)
                            bar_arrive(&x.full[slot]);
                        if (j == 0 && kv == 0)
                            copy_q();
                    }
                }
            } else {
                // 4-bit rows come through a ring of the warp's own, kRawRing K or V tiles ahead of
                // where they are decoded (from registers, the loads of one tile ahead: 3000 cycles of
                // waiting a tile).  Codes of row r, 16 bytes c: at r * 64 + (c ^ r / 2 & 3) * 16, then
                // 8 bytes of scales a row.
                const uint32_t raw0 = sm_ring + kSlots * kTileBytes + me * kRawRing * kRawBytes;
                int row = -1;                     // of the tile whose copies were issued last
                uint32_t there[3] = {0, 0, 0};    // of the tile decoded next and the two behind it
                auto issue = [&](int n, uint32_t raw) {      // K (n even) or V rows of tile n / 2
                    if (!(n & 1)) {
                        row = next_row(n >> 1);
                        there[2] = __ballot_sync(kFull, row >= 0);
                    }
                    const uint8_t *codes = (n & 1 ? a.rows.v : a.rows.k) + 16 * (lane & 3);
                    const uint8_t *scales = a.rows.scales + (size_t)(uint32_t)max(row, 0) * kScaleBytes + 8 * (n & 1);
                    const uint32_t to = raw + (lane >> 2) * kCodeBytes + (((lane & 3) ^ (lane >> 3 & 3)) << 4);
                    if (there[2] == kFull) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int from = __shfl_sync(kFull, row, 8 * i + (lane >> 2));
                            copy16(to + 8 * i * kCodeBytes, codes + (size_t)(uint32_t)from * kCodeBytes);
                        }
                    } else {
#pragma unroll 1
                        for (int i = 0; i < 4; ++i) {
                            const int from = __shfl_sync(kFull, row, 8 * i + (lane >> 2));
                            copy16(to + 8 * i * kCodeBytes, codes + (size_t)(uint32_t)max(from, 0) * kCodeBytes, from >= 0);
                        }
                    }
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(raw + 32 * kCodeBytes + 8 * lane),
                                 "l"(scales), "r"(row >= 0 ? 8 : 0)
                                 : "memory");
                };
                const int entries = 2 * u.tiles;
                // (K and V of tile 0, K of tile 1: behind each K the words of `valid` move up)
#pragma unroll
                for (int n = 0; n < kRawRing; ++n) {
                    if (n < entries)
                        issue(n, raw0 + n * kRawBytes);
                    if (n == 0)
                        there[0] = there[2];
                    if (n == 2)
                        there[1] = there[2];
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }
                uint32_t raw = raw0;
#pragma unroll 1
                for (int n = 0; n < entries; ++n) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(kRawRing - 1) : "memory");
                    __syncwarp();                 // (every lane's copies)
                    const uint32_t slot = next_slot(!(n & 1), there[0]);
                    if (!ok)
                        break;
                    // a lane decodes 32 values, c, of rows 8 t + the low three bits of its number
                    const int c = lane >> 3, low = lane & 7;
                    const uint32_t codes = raw + low * kCodeBytes + ((c ^ (low >> 1 & 3)) << 4);
                    const uint32_t scales = raw + 32 * kCodeBytes + 8 * low + 2 * c;
                    const uint32_t dst = sm_ring + slot * kTileBytes + (c >> 1) * kHalfBytes +
                                         (kCopyRows * me + low) * 128 + (((4 * (c & 1)) ^ low) << 4);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        uint32_t w[4], s2, two[2];
                        lds_words(codes + 8 * t * kCodeBytes, w);
                        asm volatile("{\n\t.reg .b16 t;\n\tld.shared.b16 t, [%1];\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
                                     : "=r"(s2)
                                     : "r"(scales + 64 * t)
                                     : "memory");
                        two[0] = __byte_perm(s2, s2, 0x1010);
                        two[1] = __byte_perm(s2, s2, 0x3232);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t y[4];
                            decode8(w[k], two[k >> 1], y);
                            sts4((dst ^ (k << 4)) + 1024 * t, y[0], y[1], y[2], y[3]);
                        }
                    }
                    arrive(&x.full[slot]);        // (with a __syncwarp: the coded rows have been read)
                    if (n == 0)
                        copy_q();
                    if (n + kRawRing < entries)
                        issue(n + kRawRing, raw);
                    if (n & 1) {                  // (the issue above was of K)
                        ++tile_no;
                        there[0] = there[1];
                        there[1] = there[2];
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    raw = raw == raw0 + (kRawRing - 1) * kRawBytes ? raw0 : raw + kRawBytes;
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
            }
            if (!ok)
                break;
            __syncwarp();
            if (lane == 0)
                free_unit();
        }
        if (flags)
            atomicOr(a.status, flags);
    } else if (warp >= kIssuer) {
        // ---- MMA issue, by one thread for each row tile: S of the next step as soon as the softmax has
        // this one's in registers, then P V of this one, so that the softmax finds its next scores
        // when it is done with these.  The tensor cores queue few MMAs, so one thread's
        // waits would leave them idle where two overlap.  (A wait
        // that gave up lets the step's MMAs go, whose results nobody uses.)
        if (elect_one()) {
            const int t = warp - kIssuer;
            uint32_t k_slot = 0, k_phase = 0, v_slot = 1, v_phase = 0;      // ring slots of the tile's K and V
            uint32_t p_buf = 0;                   // buffer of the next P V
            uint32_t p_phase = 0;                 // bit b: phase of p[t][b]
            uint32_t r_phase = 1;                 // phase of the last S that was issued
            uint32_t done_steps = 0;
            const uint32_t q = operand(sm_q + t * kTileBytes, 16);
            const uint32_t ring_k = operand(sm_ring, 16), ring_v = operand(sm_ring, kHalfBytes);
            const uint32_t col_s = 128 * t, col_p = col_s + kColP, col_o = kColO + 128 * t;
            uint64_t *const s_bar = &x.s[t], *const p_bar = x.p[t], *const o_bar = x.o[t];
            auto wait = [&](uint64_t *bar, uint32_t phase) { ok = bar_wait(bar, phase) && ok; };
            // Rows copied by cp.async are read by the MMAs through the async proxy.
            auto wait_rows = [&](uint64_t *bar, uint32_t phase) {
                wait(bar, phase);
                if (!Q4)
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            };
            auto advance = [](uint32_t &slot, uint32_t &phase) {     // two slots on
                slot += 2;
                if (slot >= kSlots) {
                    slot -= kSlots;
                    phase ^= 1;
                }
            };
            // S of a step, over the one before (which may be another unit's).
            auto issue_s = [&](uint32_t k) {
                wait(&x.r[t], r_phase);
                r_phase ^= 1;
                tmem_after();
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t o = (s >> 2) * kHalfBytes + (s & 3) * 32;
                    mma_ss<kStep, Q4>(col_s, q + (o >> 4), k + (o >> 4), s > 0);
                }
                mma_commit(s_bar);
            };
#pragma unroll 1
            for (;; ++units) {
                wait(&x.unit_there[units % kUnitRing], units / kUnitRing);
                if (!ok || unit_entry().tiles < 0)
                    break;
                const int steps = unit_entry().steps;
                wait_rows(&x.q, units);
                if (t * kTile >= unit_entry().rows) {         // the unit has no such row tile
                    bar_arrive(&x.q_free);
#pragma unroll 1
                    for (int i = 0; i < steps && ok; i += 2) {
                        wait(&x.full[k_slot], k_phase);
                        bar_arrive(&x.empty[k_slot]);
                        wait(&x.full[v_slot], v_phase);
                        bar_arrive(&x.empty[v_slot]);
                        advance(k_slot, k_phase);
                        advance(v_slot, v_phase);
                    }
                    if (!ok)
                        break;
                    free_unit();
                    continue;
                }
                wait_rows(&x.full[k_slot], k_phase);
                uint32_t k = ring_k + k_slot * (kTileBytes >> 4);
                issue_s(k);
                if (steps == 1) {
                    mma_commit(&x.empty[k_slot]);
                    mma_commit(&x.q_free);
                    advance(k_slot, k_phase);
                }
#pragma unroll 1
                for (int i = 0; i < steps && ok; ++i) {
                    const bool odd = i & 1;
                    if (i + 1 < steps) {          // S of step i + 1
                        if (odd) {
                            wait_rows(&x.full[k_slot], k_phase);
                            k = ring_k + k_slot * (kTileBytes >> 4);
                        }
                        issue_s(k + (odd ? 0 : kStep * 128 >> 4));
                        if (!odd || i + 2 == steps) {         // the tile's last one
                            mma_commit(&x.empty[k_slot]);
                            advance(k_slot, k_phase);
                        }
                        if (i + 2 == steps)
                            mma_commit(&x.q_free);
                    }
                    if (!odd)
                        wait_rows(&x.full[v_slot], v_phase);
                    const uint32_t v = ring_v + v_slot * (kTileBytes >> 4) + (odd ? kStep * 128 >> 4 : 0);
                    wait(p_bar + p_buf, p_phase >> p_buf);
                    tmem_after();
#pragma unroll
                    for (int s = 0; s < kStep / 16; ++s)
                        mma_ts<Q4>(col_o, col_p + 32 * p_buf + s * 8, v + (s * 16 * 128 >> 4), i > 0 || s > 0);
                    mma_commit(o_bar + p_buf);
                    p_phase ^= 1u << p_buf;
                    p_buf ^= 1;
                    if (odd || i + 1 == steps) {
                        mma_commit(&x.empty[v_slot]);
                        advance(v_slot, v_phase);
                    }
                    progress->tiles = ++done_steps;
                }
                if (!ok)
                    break;
                free_unit();
            }
            // No arrival of the last commits may be left when the CTA ends.
            mma_commit(&x.done[t]);
            bar_wait(&x.done[t], 0);
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---- softmax: a thread per query row of its row tile
        const int part = warp >> 2;
        const int r = tid & 127;                              // row of the row tile, and TMEM lane
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t col_s = tmem + 128 * part + lanes, col_o = tmem + kColO + 128 * part + lanes;
        uint32_t count = 0, tile_no = 0;                      // steps of this row tile; tiles of the CTA
        const uint32_t s_bar = smem_of(a.wait_test ? &x.never : &x.s[part]), s_phases = a.wait_test ? 0 : 1;
        const uint32_t r_bar = smem_of(&x.r[part]), p_bar = smem_of(&x.p[part][0]), o_bar = smem_of(&x.o[part][0]);
        auto wait_at = [&](uint32_t bar, uint32_t phase) {
            return (bool)__all_sync(kFull, bar_try(bar, phase) || bar_wait_long(bar, phase, progress, a.wait_cycles));
        };
#pragma unroll 1
        for (; next_unit(); ++units) {
            const Unit &u = unit_entry();
            const int tiles = u.tiles, steps = u.steps;
            if (part * kTile >= u.rows) {                     // the unit has no such row tile
                tile_no += tiles;
                __syncwarp();
                if (lane == 0)
                    free_unit();
                continue;
            }
            const int mine = part * kTile + r;                // row of the unit
            const bool live = mine < u.rows;
            auto row_at = [&](int i) { return u.row0 + min(i, u.rows - 1); };
            auto position_at = [&](int row) { return u.pos0 + (row >> a.g_shift); };
            // what the row sees of the unit's list of tokens: below its own place, and from the
            // window's begin on or among the first ones
            const int shift = u.first - u.low;
            const int end = position_at(row_at(mine)) + 1 + shift, low = a.window > 0 ? end - a.window : 0;
            // (of the warp's rows the first one ends first, the last one's window begins last)
            const int end0 = __shfl_sync(kFull, end, 0), low1 = __shfl_sync(kFull, low, 31);
            float sl2 = a.scale * kLog2e;
            float mref = -CUDART_INF_F, l = 0.0f;
            int t0 = u.tile0 * kTile;                         // first of the step's tokens
#pragma unroll 1
            for (int i = 0; i < steps; ++i, ++count, t0 += kStep) {
                const uint32_t buf = count & 1;
                // S of this step, and P V of the step but one before (issued before that S: over, or nearly)
                const uint32_t s_phase = count & s_phases, o_phase = (count >> 1 & 1) ^ 1;
                if (!__all_sync(kFull, bar_try(s_bar, s_phase) & bar_try(o_bar + 8 * buf, o_phase)))
                    ok = wait_at(s_bar, s_phase) && wait_at(o_bar + 8 * buf, o_phase);
                if (!ok)
                    break;
                tmem_after();
                float s[kStep];                               // the row's scores
                tmem_ld32(col_s, reinterpret_cast<uint32_t *>(s));
                tmem_ld32(col_s + 32, reinterpret_cast<uint32_t *>(s) + 32);
                if (Q4 && i == 0)                             // (written with Q, so there behind the first S)
                    sl2 *= x.q_inv[units & 1][min(mine, u.rows - 1)];
                const uint32_t *valid = &x.valid[(tile_no + (i >> 1)) % kMaskRing][2 * (i & 1)];
                uint32_t w0 = valid[0], w1 = valid[1];
                tmem_wait_ld();
                tmem_loaded(reinterpret_cast<uint32_t *>(s));
                tmem_loaded(reinterpret_cast<uint32_t *>(s) + 32);
                tmem_before();
                arrive_at(r_bar);
                // does every row of the warp see all of the step's tokens?
                const bool inside = end0 >= t0 + kStep && (t0 >= low1 || t0 + kStep <= a.sinks);
                if (!inside || (w0 & w1) != kFull) {
                    w0 &= low_bits(end - t0) & (~low_bits(low - t0) | low_bits(a.sinks - t0));
                    w1 &= low_bits(end - t0 - 32) & (~low_bits(low - t0 - 32) | low_bits(a.sinks - t0 - 32));
#pragma unroll
                    for (int k0 = 0; k0 < kStep; k0 += 16) {
                        const uint32_t m = (k0 < 32 ? w0 : w1) >> (k0 & 31);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (!(m & 1u << k))
                                s[k0 + k] = -CUDART_INF_F;
                    }
                }
                // P = 2^(x - mref).  A row's reference is its largest score at first and stays as it is until the
                // sum of a step's P passes kMostSum; then it becomes the largest score so far, O and
                // l are rescaled and P is done again.  (Rows that do not exist hold anything: not theirs.)
                float step_sum = 0.0f;
                auto probabilities = [&] {
                    // (a row that has seen nothing: any score that is not -inf gives at least 1)
                    const float off = mref == -CUDART_INF_F ? kMostFloat : -mref;
                    const float2 off2 = make_float2(off, off), sl22 = make_float2(sl2, sl2);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float2 z = __ffma2_rn(make_float2(s[32 * h + 2 * k], s[32 * h + 2 * k + 1]), sl22, off2);
                            const float2 ev = make_float2(ex2(z.x), ex2(z.y));
                            sum[k & 1] = __fadd2_rn(sum[k & 1], ev);
                            pk[k] = Q4 ? pack_f16(ev.x, ev.y) : pack_bf16(ev.x, ev.y);
                        }
                        tmem_st16(col_s + kColP + 32 * buf + 16 * h, pk);
                    }
                    step_sum = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                };
                bool grow = true, move = i == 0;
                if (!move) {
                    probabilities();
                    grow = live && !(step_sum <= (mref == -CUDART_INF_F ? 0.0f : kMostSum));
                    move = __any_sync(kFull, grow);
                }
                if (__builtin_expect(move, 0)) {
                    tmem_wait_st();                      // (P goes to the same place once more)
                    float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int k = 0; k < kStep; k += 2)
                        mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], s[k], s[k + 1]);
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                    const float mn = grow ? fmaxf(mref, top) : mref;
                    const float f = mref == mn || mref == -CUDART_INF_F ? 1.0f : ex2(mref - mn);     // (or l = 0, O = 0)
                    mref = mn;
                    if (i > 0) {
                        l *= f;
                        ok = warp_wait(&x.o[part][buf ^ 1], (count - 1) >> 1);
                        if (!ok)
                            break;
                        tmem_after();
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t ov[16];
                            tmem_ld16(col_o + 16 * c, ov);
                            tmem_wait_ld();
                            tmem_loaded16(ov);
#pragma unroll
                            for (int k = 0; k < 16; k += 2)
                                scale2(ov + k, f);
                            tmem_st16(col_o + 16 * c, ov);
                        }
                    }
                    probabilities();
                }
                l += step_sum;
                tmem_wait_st();
                tmem_before();
                arrive_at(p_bar + 8 * buf);
            }
            if (!ok)
                break;
            tile_no += tiles;
            // ---- the rows' results
            ok = warp_wait(&x.o[part][(count - 1) & 1], (count - 1) >> 1);
            if (!ok)
                break;
            tmem_after();
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            // (once more: no register holds them through the steps, and no local memory)
            const int row = row_at(opaque(mine)), p = position_at(row);
            const size_t q_row = ((size_t)u.q0 + (row >> a.g_shift)) * a.Hq + (size_t)u.h * a.G + (row & (a.G - 1));
            const bool whole = u.part < 0;
            float2 worst = make_float2(0.0f, 0.0f);           // NaN where a value is not finite
            const int q0 = u.q0, unit_row0 = u.row0, unit_rows = u.rows, unit_b = u.b, unit_h = u.h, unit_part = u.part;
            __syncwarp();
            if (lane == 0)
                free_unit();
            // A lane has a row, four lanes four rows: they turn blocks of four 16-byte pieces, so that
            // a store of the four goes to 64 bytes of one row.  (Every lane on its own: 8400 cycles
            // a unit.)
            const int row4 = part * kTile + (warp & 3) * 32 + (lane & ~3);     // first of the four rows
#pragma unroll 1
            for (int c = 0; c < (whole ? 2 : 4); ++c) {
                uint32_t y[32];
                __syncwarp();
                if (whole) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t ov[32];
                        tmem_ld32(col_o + 64 * c + 32 * half, ov);
                        tmem_wait_ld();
                        tmem_loaded(ov);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            scale2(ov + 2 * k, inv);
                            const float v0 = __uint_as_float(ov[2 * k]), v1 = __uint_as_float(ov[2 * k + 1]);
                            worst = __ffma2_rn(make_float2(0.0f, 0.0f), make_float2(v0, v1), worst);
                            y[16 * half + k] = pack_bf16(v0, v1);
                        }
                    }
                } else {
                    tmem_ld32(col_o + 32 * c, y);
                    tmem_wait_ld();
                    tmem_loaded(y);
                }
                if (whole && __any_sync(kFull, l == 0.0f)) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        y[k] = l == 0.0f ? 0u : y[k];
                }
                turn4(y, lane);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (row4 + k >= unit_rows)
                        continue;
                    const int to = unit_row0 + row4 + k;
                    uint16_t *const dst =
                        whole ? a.out + (((size_t)q0 + (to >> a.g_shift)) * a.Hq + (size_t)unit_h * a.G + (to & (a.G - 1))) *
                                            kHeadDim + 64 * c
                              : reinterpret_cast<uint16_t *>(&a.ws->prompt_o[unit_part][row4 + k][32 * c]);
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        reinterpret_cast<uint4 *>(dst)[4 * g + (lane & 3)] =
                            make_uint4(y[16 * g + 4 * k], y[16 * g + 4 * k + 1], y[16 * g + 4 * k + 2], y[16 * g + 4 * k + 3]);
                }
            }
            if (!whole && live) {
                a.ws->prompt_m[unit_part][mine] = mref;
                a.ws->prompt_l[unit_part][mine] = l;
            }
            tmem_before();
            uint32_t again = __ballot_sync(kFull, live && whole && l != 0.0f && !(worst.x + worst.y == 0.0f));
            if (again) {
                __syncwarp();                        // (the rows' stores come before the second ones)
                for (; again; again &= again - 1) {
                    const int k = __ffs(again) - 1;
                    attend_row<Q4>(a, unit_b, unit_h, __shfl_sync(kFull, p, k), __shfl_sync(kFull, (unsigned long long)q_row, k),
                                   lane, &x.progress.walked);
                }
            }
            __syncwarp();
        }
    }
    tmem_before();
    __syncthreads();
    if (x.progress.gave_up) {
        // A wait gave up: leave no copy and no MMA in flight.
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (warp >= kIssuer && elect_one()) {        // (the lane that issued them)
            mma_commit(&x.drain[warp - kIssuer]);
            bar_wait_for(&x.drain[warp - kIssuer], 0, &x.last_waits[warp], 2000000000ll);
        }
        __syncthreads();
    }
    if (tid == 0 && x.progress.gave_up)
        atomicOr(a.status, kFlagWaitTimeout);
    if (warp == kIssuer) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(x.tmem), "r"(kTmemCols)
                     : "memory");
    }
}

// Joins the parts of the units that several CTAs shared.  Block x belongs to the begin of CTA x + 1's
// range, which left a plan of the unit that it cuts (rows 0: none, or not the unit's first cut).
// A warp per query row: o = sum_s o_s 2^(m_s - m) / sum_s l_s 2^(m_s - m).
constexpr int kJoinWarps = 4, kJoinBlocks = 16;

__global__ void __launch_bounds__(32 * kJoinWarps) prompt_join_kernel(const __grid_constant__ PromptArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31, c = blockIdx.x + 1;
    const PromptJoin j = a.ws->join[c];
    if (j.rows == 0)
        return;
    // part s: CTA c - 1 + s's; its second one where its range begins with another unit
    const PromptJoin before = a.ws->join[c - 1];
    const int late = before.b != j.b || before.h != j.h || before.row0 != j.row0;
    auto part_of = [&](int s) { return 2 * (c - 1 + s) + (s == 0 ? late : 0); };
    const int parts = j.last - c + 2;
    for (int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5); r < j.rows; r += kJoinBlocks * kJoinWarps) {
        constexpr int kAhead = 4;
        float top = -CUDART_INF_F, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int s0 = 0; s0 < parts; s0 += kAhead) {
            float ms[kAhead], ls[kAhead];
            float4 x[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                ms[k] = -CUDART_INF_F;
                ls[k] = 0.0f;
                x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (s0 + k < parts) {
                    const int p = part_of(s0 + k);
                    ms[k] = a.ws->prompt_m[p][r];
                    ls[k] = a.ws->prompt_l[p][r];
                    x[k] = *reinterpret_cast<const float4 *>(&a.ws->prompt_o[p][r][4 * lane]);
                }
            }
            float mn = top;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                mn = fmaxf(mn, ms[k]);
            const float ref = mn == -CUDART_INF_F ? 0.0f : mn;
            const float keep = exp2f(top - ref);
            l *= keep;
            o.x *= keep;
            o.y *= keep;
            o.z *= keep;
            o.w *= keep;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (ls[k] == 0.0f)               // nothing of the part is seen (its sums may hold anything)
                    continue;
                const float f = ms[k] == -CUDART_INF_F ? 1.0f : exp2f(ms[k] - ref);
                l += ls[k] * f;
                o.x += x[k].x * f;
                o.y += x[k].y * f;
                o.z += x[k].z * f;
                o.w += x[k].w * f;
            }
            top = mn;
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int row = j.row0 + r;
        const size_t q_row = ((size_t)j.q0 + (row >> a.g_shift)) * a.Hq + (size_t)j.h * a.G + (row & (a.G - 1));
        const float worst = 0.0f * o.x + 0.0f * o.y + 0.0f * o.z + 0.0f * o.w;
        if (__any_sync(kFull, !(worst * inv == 0.0f))) {
            if (a.rows.scales)
                attend_row<true>(a, j.b, j.h, j.pos0 + (row >> a.g_shift), q_row, lane, nullptr);
            else
                attend_row<false>(a, j.b, j.h, j.pos0 + (row >> a.g_shift), q_row, lane, nullptr);
            continue;
        }
        uint2 y;
        y.x = pack_bf16(o.x * inv, o.y * inv);
        y.y = pack_bf16(o.z * inv, o.w * inv);
        *reinterpret_cast<uint2 *>(a.out + q_row * kHeadDim + 4 * lane) = y;
    }
}

template <bool Q4> cudaError_t launch(const PromptArgs &a, int sms, cudaStream_t stream)
{
    static std::mutex mu;
    static bool ready[64] = {false};
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !ready[dev]) {
            err = cudaFuncSetAttribute(prompt_attention_kernel<Q4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)kSmem);
            if (err != cudaSuccess)
                return err;
            if (dev >= 0 && dev < 64)
                ready[dev] = true;
        }
    }
    const int ctas = sms < kMaxPromptCtas ? sms : kMaxPromptCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, prompt_attention_kernel<Q4>, a);
    if (err != cudaSuccess || ctas < 2)
        return err;
    cfg.gridDim = dim3(ctas - 1, kJoinBlocks);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, prompt_join_kernel, a);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, int sms, cudaStream_t stream)
{
    return a.rows.scales ? launch<true>(a, sms, stream) : launch<false>(a, sms, stream);
}

}  // namespace td
