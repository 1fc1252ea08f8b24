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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
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
constexpr int kUnitRows = 2 * kTile;
constexpr int kSlots = 5;                        // ring of K and V tiles
constexpr int kMaskRing = 8;
constexpr int kSoftWarps = 8;                    // four per row tile
constexpr int kCopier = 8, kCopiers = 4;         // copy warps
constexpr int kIssuer = 12, kSched = 13;
constexpr int kThreads = 32 * 14;
constexpr int kUnitRing = 2;
constexpr int kUnitUsers = kSoftWarps + kCopiers + 1;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;                  // O of row tile t: kColO + 128 t; S: 128 t; P: 128 t + 64
constexpr size_t kSmem = (size_t)(2 + kSlots) * kTileBytes + 3 * 1024;    // + Extra

// A unit of work, as every role reads it.
struct Unit {
    int b, h;
    int q0;            // first row of q of the request
    int row0, rows;    // query rows of the request: row = token * G + head
    int pos0;          // position of the request's first new token
    int limit;         // cached tokens that some row may see: positions below this
    int low;           // and at or behind this, or below sinks
    int sink_tiles, low_tile;
    int tiles;         // of 128 tokens; -1: no more units

    __device__ int tile(int j) const { return j < sink_tiles ? j : low_tile + j - sink_tiles; }
};

// Who arrives and who waits; a wait looks at a phase's parity, so each must come when
// the phase before is over and before the one after can be.
//   full     a ring slot's use: every copy thread as its copies land, and once more each copy
//            warp, behind its word of `valid`.  The issuer waits for every one in order.
//   empty    the commit behind the MMAs that read the slot; the copy warps wait for every use.
//   q, q_free   as full and empty, per unit.
//   s[t]     S of row tile t.  Its softmax warps wait for every one; the next S is issued
//            behind P V, which needs their P.
//   p[t]     the row tile's four softmax warps; the issuer waits for every one.
//   o[t]     P V of row tile t.  The issuer waits for every one before the next S of t, which
//            overwrites its P; the softmax for the last one, or to rescale O, always
//            before it hands over the P that the next one needs.
//   unit_there, unit_free   a unit's entry, written by the scheduler and read by all others,
//            who free it when they are done with the unit.
struct Extra {
    uint64_t full[kSlots], empty[kSlots];
    uint64_t q, q_free;
    uint64_t s[2], p[2], o[2];
    uint64_t unit_there[kUnitRing], unit_free[kUnitRing];
    uint64_t drain, done, never;
    Unit unit[kUnitRing];
    alignas(16) uint32_t valid[kMaskRing][4];    // tokens of a tile that exist
    float q_inv[kUnitRing][kUnitRows];           // 4-bit rows: what a row's scores are multiplied by
    uint32_t tmem;
    Progress progress;
    Progress last_waits[kThreads / 32];
};
static_assert((2 + kSlots) * kTileBytes + sizeof(Extra) <= kSmem, "shared memory");

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

// Bits lo .. hi - 1 of 32 that start at bit `base`.
__device__ __forceinline__ uint32_t bits_of(int lo, int hi, int base)
{
    const int x = max(lo - base, 0), y = min(hi - base, 32);
    return x >= y ? 0u : (0xffffffffu >> (32 - (y - x))) << x;
}

// Four consecutive values of a cached row.
__device__ float4 row_values(const RowsArgs &c, bool v, int row, int lane)
{
    const uint8_t *x = v ? c.v : c.k;
    if (!c.scales) {
        const uint2 y = *reinterpret_cast<const uint2 *>(x + (size_t)(uint32_t)row * (kHeadDim * 2) + 8 * lane);
        return make_float4(bf_lo(y.x), bf_hi(y.x), bf_lo(y.y), bf_hi(y.y));
    }
    const uint32_t codes = *reinterpret_cast<const uint16_t *>(x + (size_t)(uint32_t)row * kCodeBytes + 2 * lane);
    const __half_raw s = __nv_cvt_fp8_to_halfraw(c.scales[(size_t)(uint32_t)row * kScaleBytes + (v ? 8 : 0) + lane / 4], __NV_E4M3);
    const float f = __half2float(__half(s));
    auto value = [&](uint32_t n) {
        const float mag = (n & 7) < 2 ? 0.5f * (n & 7) : (float)(2 + (n & 1)) * 0.5f * (float)(1 << ((n >> 1 & 3) - 1));
        return (n & 8 ? -mag : mag) * f;
    };
    return make_float4(value(codes & 15), value(codes >> 4 & 15), value(codes >> 8 & 15), value(codes >> 12));
}

// One query row by a warp, a position at a time: for rows whose tiles held values that are
// not finite, which in a product meet the zero probabilities of tokens that the row does not
// see.  Rare, and out of line.
__device__ __noinline__ void attend_row(const PromptArgs &a, int b, int h, int p, size_t q_row, int lane)
{
    const uint2 y = *reinterpret_cast<const uint2 *>(a.q + q_row * kHeadDim + 4 * lane);
    const float4 q = make_float4(bf_lo(y.x), bf_hi(y.x), bf_lo(y.y), bf_hi(y.y));
    const Range w = window_range(p + 1, a.window, a.sinks);
    float m = -CUDART_INF_F, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int t = 0; t < w.first + p + 1 - w.low; ++t) {
        const int j = t < w.first ? t : w.low + t - w.first;
        const int row = row_of(a.rows, a.Hkv, h, j, page_of(a.rows, b, j));
        if (row < 0)
            continue;
        const float4 k = row_values(a.rows, false, row, lane), v = row_values(a.rows, true, row, lane);
        float s = fmaf(q.x, k.x, fmaf(q.y, k.y, fmaf(q.z, k.z, q.w * k.w)));
#pragma unroll
        for (int d = 16; d; d >>= 1)
            s += __shfl_xor_sync(kFull, s, d);
        const float x = s * (a.scale * kLog2e), mn = fmaxf(m, x);
        const float f = safe_exp2_diff(m, mn), e = exp2f(x - (mn == -CUDART_INF_F ? 0.0f : mn));
        m = mn;
        // (a sum that is zero has nothing to keep, whatever the factor)
        l = l * f + e;
        o.x = o.x * f + e * v.x;
        o.y = o.y * f + e * v.y;
        o.z = o.z * f + e * v.z;
        o.w = o.w * f + e * v.w;
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
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    Extra &x = *reinterpret_cast<Extra *>(sm_raw + (2 + kSlots) * kTileBytes);
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
        if (tid == 0)
            atomicOr(a.status, kFlagWaitTimeout);
        return;
    }
    if (tid == 32 * kIssuer) {
        x.progress = Progress{};
        for (int i = 0; i < kThreads / 32; ++i)
            x.last_waits[i] = Progress{};
        for (int i = 0; i < kSlots; ++i) {
            bar_init(&x.full[i], 33 * kCopiers);
            bar_init(&x.empty[i], 1);
        }
        bar_init(&x.q, 32 * kCopiers);
        bar_init(&x.q_free, 1);
        for (int t = 0; t < 2; ++t) {
            bar_init(&x.s[t], 1);
            bar_init(&x.p[t], 4);
            bar_init(&x.o[t], 1);
        }
        for (int i = 0; i < kUnitRing; ++i) {
            bar_init(&x.unit_there[i], 1);
            bar_init(&x.unit_free[i], kUnitUsers);
        }
        bar_init(&x.drain, 1);
        bar_init(&x.done, 1);
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
    const uint32_t tmem = x.tmem;
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

    if (warp == kSched) {
        // ---- scheduler: units by a counter, so that the CTAs end together.  Request b's blocks of
        // 256 rows are numbers floor(cu[b] G / 256) + b and on (room for all of them; a number
        // without a block is passed over), its last ones first: they see the most tokens.
        const int64_t numbers = (int64_t)a.num_tokens * a.G / kUnitRows + a.B;
        const int64_t total = numbers * a.Hkv;
        auto start_of = [&](int b) { return min(max(a.cu_new[b], 0), a.num_tokens); };
        auto number_of = [&](int b) { return (int64_t)start_of(b) * a.G / kUnitRows + b; };
#pragma unroll 1
        while (ok) {
            Unit u{};
            u.tiles = -1;
            uint32_t bad = 0;
#pragma unroll 1
            for (;;) {
                uint32_t at = 0;
                if (lane == 0)
                    at = atomicAdd(&a.ws->units, 1u);
                at = __shfl_sync(kFull, at, 0);
                if (at >= total)
                    break;
                const int64_t number = at / (uint32_t)a.Hkv;
                int lo = 0, hi = a.B;             // the last request that begins at or before the number
                while (hi - lo > 1) {
                    const int step = (hi - lo + 31) / 32, b = lo + lane * step;
                    const int n = __popc(__ballot_sync(kFull, b < hi && (lane == 0 || number_of(b) <= number)));
                    lo += (n - 1) * step;
                    hi = min(hi, lo + step);
                }
                const int q0 = start_of(lo), count = max(0, start_of(lo + 1) - q0);
                const int blocks = (int)(((int64_t)count * a.G + kUnitRows - 1) / kUnitRows);
                const int64_t block = number - number_of(lo);
                if (block < 0 || block >= blocks)
                    continue;
                u.b = lo;
                u.h = at % (uint32_t)a.Hkv;
                u.q0 = q0;
                u.row0 = (blocks - 1 - (int)block) * kUnitRows;
                u.rows = min(count * a.G - u.row0, kUnitRows);
                const int n = seq_len_of(a.seq_lens, lo, a.Nmax, bad);
                if (count > n)
                    bad |= kFlagSeqLenOutOfRange;
                u.pos0 = n - count;               // (below zero: those tokens see nothing)
                const int p0 = u.pos0 + (u.row0 >> a.g_shift);
                const int p1 = u.pos0 + ((u.row0 + u.rows - 1) >> a.g_shift);
                u.limit = max(p1 + 1, 0);
                u.low = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
                u.low_tile = u.low / kTile;
                u.sink_tiles = min((min(a.sinks, u.low) + kTile - 1) / kTile, u.low_tile);
                u.tiles = u.sink_tiles + max(1, (u.limit + kTile - 1) / kTile - u.low_tile);
                break;
            }
            if (bad && lane == 0)
                atomicOr(a.status, bad);
            if (units >= kUnitRing)
                ok = warp_wait(&x.unit_free[units % kUnitRing], units / kUnitRing - 1);
            if (!ok)
                break;
            if (lane == 0) {
                x.unit[units % kUnitRing] = u;
                bar_arrive(&x.unit_there[units % kUnitRing]);
            }
            __syncwarp();
            ++units;
            if (u.tiles < 0)
                break;
        }
    } else if (warp >= kCopier && warp < kCopier + kCopiers) {
        // ---- copy warps: a unit's Q, then its K and V tiles, 32 rows of each per warp
        const int me = warp - kCopier;
        uint32_t e = 0;                           // ring entries begun
        uint32_t flags = 0;
        uint32_t tile_no = 0;
#pragma unroll 1
        for (; next_unit(); ++units) {
            const Unit u = unit_entry();
            // the row of this lane's token of tile j; a token that no row of the unit sees is
            // none (zeros: no value of it meets a zero probability)
            auto position = [&](int j) {
                const int p = u.tile(j) * kTile + 32 * me + lane;
                return j < u.tiles && p < u.limit && (p >= u.low || p < a.sinks) ? p : -1;
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
            int p0 = position(0), p1 = position(1);
            int pg0 = page(p0), pg1 = page(p1);
            if (units > 0)
                ok = warp_wait(&x.q_free, units - 1);
            if (!ok)
                break;
            {   // Q: half a warp per row of 256 bytes
                const int c = lane & 15;
                const uint16_t *src = a.q + ((size_t)u.q0 * a.Hq + (size_t)u.h * a.G) * kHeadDim + c * 8;
                const uint32_t dst = sm_q + (c >> 3) * kHalfBytes;
#pragma unroll 4
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
                            x.q_inv[units % kUnitRing][r] = __uint_as_float((uint32_t)(127 - up) << 23);
                    }
                }
                if constexpr (!Q4) {
                    copies_arrive(&x.q);
                } else {
                    __syncwarp();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    bar_arrive(&x.q);
                }
            }
#pragma unroll 1
            for (int j = 0; j < u.tiles; ++j, ++tile_no) {
                const int row = find(p0, pg0);
                p0 = p1;
                pg0 = pg1;
                p1 = position(j + 2);
                pg1 = page(p1);
                const uint32_t there = __ballot_sync(kFull, row >= 0);
                if constexpr (!Q4) {
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++e) {
                        const uint32_t slot = e % kSlots, use = e / kSlots;
                        if (use > 0)
                            ok = warp_wait(&x.empty[slot], use - 1);
                        if (!ok)
                            break;
                        if (kv == 0 && lane == 0)
                            x.valid[tile_no % kMaskRing][me] = there;
                        const int c = lane & 15;
                        const uint8_t *src = (kv ? a.rows.v : a.rows.k) + c * 16;
                        const uint32_t dst = sm_ring + slot * kTileBytes + (c >> 3) * kHalfBytes + 32 * me * 128;
#pragma unroll 4
                        for (int r = lane >> 4; r < 32; r += 2) {
                            const int from = __shfl_sync(kFull, row, r);
                            copy16(dst + r * 128 + (((c ^ r) & 7) << 4),
                                   src + (size_t)(uint32_t)max(from, 0) * (kHeadDim * 2), from >= 0);
                        }
                        copies_arrive(&x.full[slot]);
                        if (lane == 0)
                            bar_arrive(&x.full[slot]);
                    }
                } else {
                    // a lane decodes 32 values (16 bytes, two scales) of four rows
                    const int c = lane >> 3;
                    uint4 w[2][4];
                    uint32_t sc[2][4];
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const int from = __shfl_sync(kFull, row, 8 * t + (lane & 7));
                            const size_t at = (uint32_t)max(from, 0);
                            w[kv][t] = *reinterpret_cast<const uint4 *>((kv ? a.rows.v : a.rows.k) + at * kCodeBytes + 16 * c);
                            sc[kv][t] = from >= 0 ? *reinterpret_cast<const uint16_t *>(a.rows.scales + at * kScaleBytes + 8 * kv + 2 * c) : 0;
                        }
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv, ++e) {
                        const uint32_t slot = e % kSlots, use = e / kSlots;
                        if (use > 0)
                            ok = warp_wait(&x.empty[slot], use - 1);
                        if (!ok)
                            break;
                        if (kv == 0 && lane == 0)
                            x.valid[tile_no % kMaskRing][me] = there;
                        const uint32_t dst = sm_ring + slot * kTileBytes + (c >> 1) * kHalfBytes;
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const int r = 32 * me + 8 * t + (lane & 7);
                            uint32_t s2, two[2];
                            asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
                                : "=r"(s2)
                                : "r"(sc[kv][t]));
                            two[0] = __byte_perm(s2, s2, 0x1010);
                            two[1] = __byte_perm(s2, s2, 0x3232);
                            const uint32_t words[4] = {w[kv][t].x, w[kv][t].y, w[kv][t].z, w[kv][t].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                uint32_t y[4];
                                decode8(words[k], two[k >> 1], y);
                                const int chunk = 4 * (c & 1) + k;      // of the row's half
                                sts4(dst + r * 128 + (((chunk ^ r) & 7) << 4), y[0], y[1], y[2], y[3]);
                            }
                        }
                        __syncwarp();
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        bar_arrive_n(&x.full[slot], lane == 0 ? 2 : 1);
                    }
                }
                if (!ok)
                    break;
            }
            if (!ok)
                break;
            __syncwarp();
            if (lane == 0)
                free_unit();
        }
        if (flags)
            atomicOr(a.status, flags);
    } else if (warp == kIssuer) {
        // ---- MMA issue, by one thread
        if (elect_one()) {
            uint32_t e = 0;                       // ring entry of the unit's first K tile
            uint32_t pv[2] = {0, 0};              // P V issued so far, per row tile
            uint32_t done_tiles = 0;
            auto wait = [&](uint64_t *bar, uint32_t phase) {
                ok = ok && bar_wait(bar, phase);
                return ok;
            };
            auto proxy_fence = [] { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); };
            auto wait_full = [&](uint32_t entry) {
                wait(&x.full[entry % kSlots], entry / kSlots);
                proxy_fence();
                return ok;
            };
#pragma unroll 1
            for (;; ++units) {
                wait(&x.unit_there[units % kUnitRing], units / kUnitRing);
                if (!ok)
                    break;
                const int tiles = unit_entry().tiles, parts = unit_entry().rows > kTile ? 2 : 1;
                if (tiles < 0)
                    break;
                auto issue_s = [&](int t, int j) {
                    // P V before has read the P that lies over this S (and its softmax the S before)
                    if (pv[t] > 0 && !wait(&x.o[t], pv[t] - 1))
                        return;
                    tmem_after();
                    const uint32_t q = operand(sm_q + t * kTileBytes, 16);
                    const uint32_t k = operand(sm_ring + (e + 2 * j) % kSlots * kTileBytes, 16);
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t o = (s >> 2) * kHalfBytes + (s & 3) * 32;
                        mma_ss<kTile, Q4>(tmem + 128 * t, q + (o >> 4), k + (o >> 4), s > 0);
                    }
                    mma_commit(&x.s[t]);
                    if (t == parts - 1) {
                        mma_commit(&x.empty[(e + 2 * j) % kSlots]);
                        if (j == tiles - 1)
                            mma_commit(&x.q_free);
                    }
                };
                if (!wait(&x.q, units))
                    break;
                proxy_fence();
                if (!wait_full(e))
                    break;
                for (int t = 0; ok && t < parts; ++t)
                    issue_s(t, 0);
#pragma unroll 1
                for (int j = 0; ok && j < tiles; ++j) {
#pragma unroll 1
                    for (int t = 0; ok && t < parts; ++t) {
                        const uint32_t entry = e + 2 * j + 1;
                        if (t == 0 && !wait_full(entry))
                            break;
                        if (!wait(&x.p[t], pv[t]))
                            break;
                        tmem_after();
                        const uint32_t v = operand(sm_ring + entry % kSlots * kTileBytes, kHalfBytes);
#pragma unroll
                        for (int s = 0; s < kTile / 16; ++s)
                            mma_ts<Q4>(tmem + kColO + 128 * t, tmem + 128 * t + 64 + s * 8, v + (s * 16 * 128 >> 4),
                                       j > 0 || s > 0);
                        mma_commit(&x.o[t]);
                        ++pv[t];
                        if (t == parts - 1)
                            mma_commit(&x.empty[entry % kSlots]);
                        if (j + 1 < tiles) {
                            if (t == 0 && !wait_full(entry + 1))
                                break;
                            issue_s(t, j + 1);
                        }
                    }
                    progress->tiles = ++done_tiles;
                }
                if (!ok)
                    break;
                e += 2 * tiles;
                free_unit();
            }
            // No arrival of the last commits may be left when the CTA ends.
            mma_commit(&x.done);
            bar_wait(&x.done, 0);
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ---- softmax: a thread per query row of its row tile
        const int part = warp >> 2;
        const int r = tid & 127;                              // row of the row tile, and TMEM lane
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t col_s = tmem + 128 * part + lanes, col_p = col_s + 64, col_o = tmem + kColO + 128 * part + lanes;
        uint32_t count = 0, tile_no = 0;                      // tiles of this row tile; of the CTA
#pragma unroll 1
        for (; next_unit(); ++units) {
            const Unit &u = unit_entry();
            const int tiles = u.tiles;
            if (part * kTile >= u.rows) {                     // the unit has no such row tile
                tile_no += tiles;
                __syncwarp();
                if (lane == 0)
                    free_unit();
                continue;
            }
            const int mine = part * kTile + r;                // row of the unit
            const bool live = mine < u.rows;
            const int row = u.row0 + min(mine, u.rows - 1);
            const int p = u.pos0 + (row >> a.g_shift);        // position
            const int low = a.window > 0 ? p - a.window + 1 : 0;
            float sl2 = a.scale * kLog2e;
            float mref = -CUDART_INF_F, l = 0.0f;
#pragma unroll 1
            for (int j = 0; j < tiles; ++j, ++count, ++tile_no) {
                ok = warp_wait(a.wait_test ? &x.never : &x.s[part], a.wait_test ? 0 : count);
                if (!ok)
                    break;
                tmem_after();
                if (Q4 && j == 0)                             // (written with Q, so there behind the first S)
                    sl2 *= x.q_inv[units % kUnitRing][min(mine, u.rows - 1)];
                uint32_t seen[4];
                lds_words(smem_of(x.valid[tile_no % kMaskRing]), seen);
                const int t0 = u.tile(j) * kTile;
                // does every row of the warp see the whole tile?
                const bool inside = p >= t0 + kTile - 1 && (t0 >= low || t0 + kTile <= a.sinks);
                if (!__all_sync(kFull, inside)) {
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        seen[w] &= bits_of(0, p + 1 - t0, 32 * w) &
                                   (bits_of(low - t0, kTile, 32 * w) | bits_of(0, a.sinks - t0, 32 * w));
                }
                // The row's scores pass through 64 registers, in blocks of 64 tokens: both
                // for the maximum, then the second and again the first for the exponentials.
                float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
                float2 off2 = make_float2(0.0f, 0.0f);
                float2 sum[2] = {off2, off2};
#pragma unroll 1
                for (int pass = 0; pass < 3; ++pass) {
                    const int block = pass & 1;
                    const uint32_t w0 = block ? seen[2] : seen[0], w1 = block ? seen[3] : seen[1];
                    float s[64];
                    __syncwarp();
                    tmem_ld32(col_s + 64 * block, reinterpret_cast<uint32_t *>(s));
                    tmem_ld32(col_s + 64 * block + 32, reinterpret_cast<uint32_t *>(s) + 32);
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
                    if (pass < 2) {
#pragma unroll
                        for (int k = 0; k < 64; k += 2)
                            mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], s[k], s[k + 1]);
                    }
                    if (pass == 1) {
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
                        if (mref == -CUDART_INF_F)
                            mref = top;              // nothing summed so far: l = 0 and O = 0
                        // The running maximum lags until a row exceeds it by 2^8: the
                        // probabilities stay below 2^8 and O is rescaled rarely.
                        const bool grow = j > 0 && top > mref + 8.0f;
                        if (__any_sync(kFull, grow)) {
                            ok = warp_wait(&x.o[part], count - 1);
                            if (!ok)
                                break;
                            tmem_after();
                            const float mn = grow ? top : mref;
                            const float f = grow ? ex2(mref - mn) : 1.0f;
                            mref = mn;
                            l *= f;
#pragma unroll 1
                            for (int c = 0; c < 4; ++c) {
                                uint32_t ov[32];
                                tmem_ld32(col_o + 32 * c, ov);
                                tmem_wait_ld();
                                tmem_loaded(ov);
#pragma unroll
                                for (int k = 0; k < 32; k += 2)
                                    scale2(ov + k, f);
                                tmem_st32(col_o + 32 * c, ov);
                            }
                        }
                        const float off = mref == -CUDART_INF_F ? 0.0f : -mref;
                        off2 = make_float2(off, off);
                    }
                    if (pass >= 1) {
                        const float2 sl22 = make_float2(sl2, sl2);
                        uint32_t pk[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float2 z = __ffma2_rn(make_float2(s[2 * k], s[2 * k + 1]), sl22, off2);
                            const float2 ev = make_float2(ex2(z.x), ex2(z.y));
                            sum[k & 1] = __fadd2_rn(sum[k & 1], ev);
                            pk[k] = Q4 ? pack_f16(ev.x, ev.y) : pack_bf16(ev.x, ev.y);
                        }
                        // (over scores of the second block, which have been read)
                        tmem_st32(col_p + 32 * block, pk);
                    }
                }
                if (!ok)
                    break;
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
                // P V of the tile before is waited for before this P goes: no phase is missed
                if (j == tiles - 1 && j > 0)
                    ok = warp_wait(&x.o[part], count - 1);
                if (!ok)
                    break;
                tmem_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(&x.p[part]);
            }
            if (!ok)
                break;
            // ---- the rows' results
            ok = warp_wait(&x.o[part], count - 1);
            if (!ok)
                break;
            tmem_after();
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const size_t q_row = ((size_t)u.q0 + (row >> a.g_shift)) * a.Hq + (size_t)u.h * a.G + (row & (a.G - 1));
            float worst = 0.0f;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t ov[32];
                __syncwarp();
                tmem_ld32(col_o + 32 * c, ov);
                tmem_wait_ld();
                tmem_loaded(ov);
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    scale2(ov + 2 * k, inv);
                    const float v0 = __uint_as_float(ov[2 * k]), v1 = __uint_as_float(ov[2 * k + 1]);
                    worst = fmaf(0.0f, v0, fmaf(0.0f, v1, worst));      // NaN where one is not finite
                    y[k] = l == 0.0f ? 0u : pack_bf16(v0, v1);
                }
                if (live) {
                    uint4 *dst = reinterpret_cast<uint4 *>(a.out + q_row * kHeadDim + 32 * c);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dst[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
                }
            }
            tmem_before();
            uint32_t again = __ballot_sync(kFull, live && l != 0.0f && !(worst == 0.0f));
            if (again) {
                __syncwarp();                        // (the rows' stores come before the second ones)
                for (; again; again &= again - 1) {
                    const int k = __ffs(again) - 1;
                    attend_row(a, u.b, u.h, __shfl_sync(kFull, p, k), __shfl_sync(kFull, (unsigned long long)q_row, k), lane);
                }
            }
            __syncwarp();
            if (lane == 0)
                free_unit();
        }
    }
    tmem_before();
    __syncthreads();
    if (x.progress.gave_up) {
        // A wait gave up: leave no copy and no MMA in flight.
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (warp == kIssuer && elect_one()) {        // (the lane that issued them)
            mma_commit(&x.drain);
            bar_wait_for(&x.drain, 0, &x.last_waits[warp], 2000000000ll);
        }
        __syncthreads();
    }
    if (tid == 0) {
        if (x.progress.gave_up)
            atomicOr(a.status, kFlagWaitTimeout);
        // The last CTA to end leaves the counters as it found them.
        __threadfence();
        if (atomicAdd(&a.ws->done, 1u) == gridDim.x - 1) {
            a.ws->units = 0;
            a.ws->done = 0;
        }
    }
    if (warp == kIssuer) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                     : "memory");
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
    const int64_t units = ((int64_t)a.num_tokens * a.G / kUnitRows + a.B) * a.Hkv;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units < sms ? units : sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prompt_attention_kernel<Q4>, a);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs &a, int sms, cudaStream_t stream)
{
    return a.rows.scales ? launch<true>(a, sms, stream) : launch<false>(a, sms, stream);
}

}  // namespace td
