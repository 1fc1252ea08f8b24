// td_cache_attn.cu -- attention of one new token per request over a small cache:
// a window with sinks, rows of 16 or of 4 bits, a persisted index set; and the sums
// of its probabilities per cached position.
//
// Request b, KV head g, its G query heads h, positions S (a window with the first
// tokens, everything, or an index set):
//     x_j = scale q_h . K_j,   out_h = sum_{j in S} softmax(x)_j V_j   (0 for empty S)
// in one pass with a running maximum m, denominator l and output o per head.
//
// A 4-bit value is code * scale, a code of 0 .5 1 1.5 2 3 4 6 with a sign (e2m1) and an e4m3
// scale for 16 of them: 2 + 4 significant bits between 2^-10 and 2688, so fp16 holds
// it exactly and the products below see the cached values themselves.
//
// Both products run on mma.sync m16n8k16: a KV head has at most 8 query heads here, an
// eighth of a tcgen05 tile's rows, and the operands come out of registers, where
// 4-bit rows have to be decoded anyway (a tcgen05 operand would go through shared or
// tensor memory first).  S: 16 tokens x 8 heads, dims summed; O: dims x 8 heads,
// tokens summed.  The order in which a sum takes its terms is free, so a lane's dims are
// those that its loads bring: 16 bytes of a K row, of V rows 16 (8 of a 4-bit row, the
// dims of one scale).  P turns from S's layout to the second product's by a transposing
// move of 8 x 8 blocks.
//
// Measured on GB300 (a call in a graph), 32 requests of 8K .. 16K tokens, 32 query / 8 KV heads:
//   window 4096, 16-bit rows    85 us, 6.3 TB/s: bound by memory
//   everything, 4-bit rows      95 us, 4.8 TB/s: no unit is at its limit (issue slots 61%, ALU 53%, DRAM 59%).
//                              Of a warp's time 9% are waits for memory, 18% issue, 23% fixed latencies,
//                              21% another warp issues, 17% the conversions' pipe is busy: 3.5
//                              warps per scheduler, whose instructions follow on one another
//   a set of 2048 of 32K tokens, 4 requests, 4-bit rows: 10.7 us, of which two thirds are one
//                              chain of loads (length, set, page, row) and the join
//   weights, 1025 .. 4224 tokens: 70 us with the second kernel; 3 requests of 257 .. 2050: 15.5
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include <mutex>

#include "td_attn_common.cuh"
#include "td_cache.h"

namespace td {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kJoinCost = 30.0f;
constexpr int kHeads = 8;             // columns of the products; heads behind G are zero

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel)
{
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 block of 16-bit values held as mma fragments.
__device__ __forceinline__ uint32_t turned(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Loads of rows, which are read once: no L1 allocation.  Zeros where `there` is false.
__device__ __forceinline__ uint4 load16(const void *p, bool there = true)
{
    uint4 r;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
                 "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
                 "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p), "r"((uint32_t)there));
    return r;
}

// Four codes' worth of halves: two bytes of codes (those of byte `at` and at + 1 of x) as
// two pairs of fp16 values, the low half of a byte first.
__device__ __forceinline__ void decode2(uint32_t x, int at, uint32_t &lo, uint32_t &hi)
{
    if (at == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(x));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, c;\n\tcvt.rn.f16x2.e2m1x2 %1, d;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(x));
}

// Two e4m3 scales (low 16 bits of x) as fp16.
__device__ __forceinline__ uint32_t scale_pair(uint32_t x)
{
    uint32_t s;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(s) : "r"(x));
    return s;
}

// The same, each twice.
__device__ __forceinline__ void scales2(uint32_t x, uint32_t &s0, uint32_t &s1)
{
    const uint32_t s = scale_pair(x);
    s0 = prmt(s, s, 0x1010);
    s1 = prmt(s, s, 0x3232);
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_b16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// Rows of 16 tokens of a warp: lane (r, c) = (lane / 4, lane % 4) holds of K the tokens r and
// r + 8, of V the tokens 2c, 2c + 1, 2c + 8 and 2c + 9.
template <bool Q4> struct Tokens;

// 16 bits.  K: dims 8 (c + 4 i) .. + 7 in word group i; V: dims 8 r .. + 7 and 64 + 8 r .. + 7.
template <> struct Tokens<false> {
    uint4 k[2][4], v[4][2];

    __device__ void load_k(const RowsArgs &a, int r, int c, const int (&row)[2])
    {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t *p = a.k + (size_t)(uint32_t)max(row[t], 0) * (kHeadDim * 2) + 16 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                k[t][i] = load16(p + 64 * i);
        }
    }
    __device__ void load_v(const RowsArgs &a, int r, int c, const int (&row)[4])
    {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint8_t *p = a.v + (size_t)(uint32_t)max(row[t], 0) * (kHeadDim * 2) + 16 * r;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[t][i] = load16(p + 128 * i, row[t] >= 0);    // P of such a token is zero; V has to be finite
        }
    }
    __device__ void s(float (&d)[4], const uint32_t (&q)[16]) const
    {
        float odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mma<false>(d, k[0][i].x, k[1][i].x, k[0][i].y, k[1][i].y, q[4 * i], q[4 * i + 1]);
            mma<false>(odd, k[0][i].z, k[1][i].z, k[0][i].w, k[1][i].w, q[4 * i + 2], q[4 * i + 3]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            d[e] += odd[e];
    }
    __device__ static uint32_t word(const uint4 (&x)[2], int i)
    {
        const uint4 &y = x[i >> 2];
        return (i & 3) == 0 ? y.x : (i & 3) == 1 ? y.y : (i & 3) == 2 ? y.z : y.w;
    }
    // P as two bf16 terms, 16 bits together, so that the result has the accuracy of fp32
    // sums behind its one rounding.  (p[t]: of token r + 8 t, heads 2c and 2c + 1.)
    __device__ void pv(float (&o)[8][4], const float (&p)[2][2]) const
    {
        uint32_t b[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t hi = pack_b16(p[t][0], p[t][1]);
            b[0][t] = turned(hi);
            b[1][t] = turned(pack_b16(p[t][0] - bf_lo(hi), p[t][1] - bf_hi(hi)));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w0 = word(v[0], i), w1 = word(v[1], i), w2 = word(v[2], i), w3 = word(v[3], i);
            const uint32_t a0 = prmt(w0, w1, 0x5410), a1 = prmt(w0, w1, 0x7632);
            const uint32_t a2 = prmt(w2, w3, 0x5410), a3 = prmt(w2, w3, 0x7632);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                mma<false>(o[i], a0, a1, a2, a3, b[k][0], b[k][1]);
        }
    }
    __device__ static int dim(int i, int r) { return (i < 4 ? 8 * r : 64 + 8 * r) + 2 * (i & 3); }
    __device__ static int qdim(int c, int w) { return 8 * (c + 4 * (w >> 2)) + 2 * (w & 3); }   // of q word w
};

// 4 bits.  K: dims 32 c .. + 31, two scales; V: dims 16 r .. + 15, one scale.  The rows of 32
// tokens come through shared memory (a warp's own ring): K codes, 64 bytes a token; V codes, whose
// 16-byte pieces q of token t lie at place (t & 1) * 4 + q ^ (t / 2 & 3) * 2 of their two tokens'
// 128 bytes, so that a half warp's loads fall into all banks; the tokens' 16 bytes of scales.
constexpr int kStageTokens = 32;
constexpr int kStageV = kStageTokens * kCodeBytes, kStageScales = 2 * kStageV;
constexpr int kStageValid = kStageScales + kStageTokens * kScaleBytes;      // which tokens there are
constexpr int kStageBytes = kStageValid + 16;
constexpr int kStages = 3;

__device__ __forceinline__ uint32_t v_place(int t, int q) { return (t >> 1) * 128 + ((((t & 1) << 2) + q) ^ ((t >> 1 & 3) << 1)) * 16; }

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

template <> struct Tokens<true> {
    uint32_t k[2][4];
    uint2 v[4];
    uint32_t ks[2], vs[4];

    // The rows of a stage: lane's own token's is `row`, -1: none (zeros).
    __device__ static void fill(const RowsArgs &a, uint32_t stage, int row, int lane)
    {
        const int q = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 8 * i + (lane >> 2), from = __shfl_sync(kFull, row, t);
            const size_t at = (size_t)(uint32_t)max(from, 0) * kCodeBytes + 16 * q;
            copy16(stage + t * kCodeBytes + 16 * q, a.k + at, from >= 0);
            copy16(stage + kStageV + v_place(t, q), a.v + at, from >= 0);
        }
        copy16(stage + kStageScales + lane * kScaleBytes, a.scales + (size_t)(uint32_t)max(row, 0) * kScaleBytes, row >= 0);
        const uint32_t there = __ballot_sync(kFull, row >= 0);
        if (lane == 0)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(stage + kStageValid), "r"(there) : "memory");
    }
    __device__ void load_k(uint32_t stage, int u, int r, int c)
    {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int tok = 16 * u + 8 * t + r;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(k[t][0]), "=r"(k[t][1]), "=r"(k[t][2]), "=r"(k[t][3])
                         : "r"(stage + tok * kCodeBytes + 16 * c)
                         : "memory");
            asm volatile("{\n\t.reg .b16 t;\n\tld.shared.b16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}"
                         : "=r"(ks[t])
                         : "r"(stage + kStageScales + tok * kScaleBytes + 2 * c)
                         : "memory");
        }
    }
    __device__ void load_v(uint32_t stage, int u, int r, int c)
    {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int tok = 16 * u + 2 * c + (t & 1) + 8 * (t >> 1);
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                         : "=r"(v[t].x), "=r"(v[t].y)
                         : "r"(stage + kStageV + v_place(tok, r >> 1) + 8 * (r & 1))
                         : "memory");
            asm volatile("ld.shared.u8 %0, [%1];"
                         : "=r"(vs[t])
                         : "r"(stage + kStageScales + tok * kScaleBytes + 8 + r)
                         : "memory");
        }
    }
    __device__ void s(float (&d)[4], const uint32_t (&q)[16]) const
    {
        uint32_t sc[2][2];
        scales2(ks[0], sc[0][0], sc[0][1]);
        scales2(ks[1], sc[1][0], sc[1][1]);
        float odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t x[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                decode2(k[t][j >> 1], 2 * (j & 1), x[t][0], x[t][1]);
                x[t][0] = mul2(x[t][0], sc[t][j >> 2]);
                x[t][1] = mul2(x[t][1], sc[t][j >> 2]);
            }
            mma<true>((j & 1) ? odd : d, x[0][0], x[1][0], x[0][1], x[1][1], q[2 * j], q[2 * j + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            d[e] += odd[e];
    }
    // P in fp16: half a step is 2^-12 of a probability, an eighth of the output's own
    // rounding (below 2^-14 of the largest, an absolute 2^-25).
    __device__ void pv(float (&o)[8][4], const float (&p)[2][2]) const
    {
        // Two tokens' codes of a dim meet in a byte (lower token low) before they are converted, with the
        // two tokens' scales.
        const uint32_t sc[2] = {scale_pair(vs[0] | vs[1] << 8), scale_pair(vs[2] | vs[3] << 8)};
        const uint32_t b0 = turned(pack_f16(p[0][0], p[0][1])), b1 = turned(pack_f16(p[1][0], p[1][1]));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t x[2][2][4];                      // token pair, even and odd dims, dims / 2
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                constexpr uint32_t low = 0x0f0f0f0f;
                const uint32_t w0 = h ? v[2 * t].y : v[2 * t].x, w1 = h ? v[2 * t + 1].y : v[2 * t + 1].x;
                const uint32_t codes[2] = {(w0 & low) | (w1 << 4 & ~low), (w0 >> 4 & low) | (w1 & ~low)};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    decode2(codes[e], 0, x[t][e][0], x[t][e][1]);
                    decode2(codes[e], 2, x[t][e][2], x[t][e][3]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        x[t][e][k] = mul2(x[t][e][k], sc[t]);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                mma<true>(o[4 * h + k], x[0][0][k], x[0][1][k], x[1][0][k], x[1][1][k], b0, b1);
        }
    }
    __device__ static int dim(int i, int r) { return 16 * r + 2 * i; }
    __device__ static int qdim(int c, int w) { return 32 * c + 2 * w; }
};

// What a CTA does: an equal, contiguous range of the batch's groups of tokens, unit
// (request, KV head) after unit, so that the longest request decides nothing.  A unit that
// several CTAs share is joined by the last of them to come.  A unit without tokens
// has one group, of which no token exists: its result is zero.
struct Seen {
    int n, count, groups;
    Range w;
};

template <int MODE, int GT> __device__ __forceinline__ Seen seen_of(const CacheAttnArgs &a, int b, uint32_t &bad)
{
    Seen s;
    s.n = seq_len_of(a.seq_lens, b, a.Nmax, bad);
    s.w = window_range(s.n, a.window, a.sinks);
    s.count = MODE == 1 ? a.top_k : s.n - s.w.low + s.w.first;
    s.groups = max(1, (s.count + GT - 1) / GT);
    return s;
}

// MODE 0: a window or everything; 1: an index set; 2: everything, the logits are kept.
// U: 16-token blocks that a warp takes at a time (4 bits: a stage's two).
template <bool Q4, int MODE, int U, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS) cache_attention_kernel(const __grid_constant__ CacheAttnArgs a)
{
    constexpr int GT = 16 * U;
    using Block = Tokens<Q4>;
    __shared__ int sm_sums[kWarps];
    __shared__ int sm_start[3];                   // b, KV head, group that the CTA's range starts at
    __shared__ float sm_m[kWarps][kHeads], sm_l[kWarps][kHeads];
    __shared__ int sm_last;
    // Rows of 16 bits: what a unit's end needs again, so that no register holds it through the loop over the unit's
    // groups (there is none to spare, and no local memory).  The last one is read behind the unit's
    // last barrier: units take two words in turn.
    __shared__ volatile int sm_per, sm_stop, sm_begin, sm_end, sm_done[2];
    // The warps' outputs; over 4-bit rows in their rings, which are empty by then.
    extern __shared__ __align__(128) unsigned char sm_raw[];
    constexpr int kPerWarp = Q4 ? kStages * kStageBytes : kHeads * kHeadDim * (int)sizeof(float);
    auto sm_o = [&](int w, int hd) { return reinterpret_cast<float *>(sm_raw + w * kPerWarp) + hd * kHeadDim; };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int r = lane >> 2, c = lane & 3;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm_raw) + warp * kPerWarp;
    pdl_wait();

    // ---- the CTA's range: requests in equal runs per thread, prefix sums
    uint32_t bad = 0;
    int total = 0, per;
    {
        const int run = (a.B + kThreads - 1) / kThreads;
        const int b0 = min(tid * run, a.B), b1 = min(b0 + run, a.B);
        int mine = 0, last = 0;                   // groups of a KV head: all requests', the last one's
        for (int b = b0; b < b1; ++b) {
            last = seen_of<MODE, GT>(a, b, bad).groups;
            mine += last * a.Hkv;
        }
        if (bad && blockIdx.x == 0)
            atomicOr(a.status, bad);
        bad = 0;
        int inc = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, d);
            if (lane >= d)
                inc += y;
        }
        if (lane == 31)
            sm_sums[warp] = inc;
        __syncthreads();
        int at = inc - mine;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp)
                at += sm_sums[i];
            total += sm_sums[i];
        }
        // Few groups for many SMs: a part more costs the join (60 ns of one CTA), a group more each warp
        // (1 to 2 us), so that sqrt(groups of a unit / kJoinCost) groups a warp cost the least; no more
        // than one unit has.  (1 x 16000 tokens, one KV head: 11.4 us, a group a warp 26.3; 4-bit sets of
        // 2048 10.7 and 12.0; 1 x 16 tokens, 8 KV heads: 3.9, four units a CTA 10.5.)
        const int unit = max((int)((uint32_t)total / (uint32_t)(a.B * a.Hkv)), 1);
        const int least = kWarps * max((int)(sqrtf((float)unit / kJoinCost) + 0.5f), 1);
        per = max(min(least, unit), (int)((uint32_t)(total + gridDim.x - 1) / gridDim.x));
        const int64_t start = (int64_t)blockIdx.x * per;
        if (start < total && at <= start && start < at + mine) {
            for (int b = b0; b < b1; ++b) {
                const int g = run == 1 ? last : seen_of<MODE, GT>(a, b, bad).groups;
                if (start < at + (int64_t)g * a.Hkv) {
                    sm_start[0] = b;
                    sm_start[1] = (int)(start - at) / g;
                    sm_start[2] = (int)(start - at) % g;
                    break;
                }
                at += g * a.Hkv;
            }
        }
        if (!Q4 && tid == 0) {
            sm_per = per;
            sm_stop = (int)min(start + per, (int64_t)total);
        }
        __syncthreads();
        if (start >= total)
            return;
    }
    int at = blockIdx.x * per;                    // groups done, in the whole batch's order
    int stop = min(at + per, total);
    int b = sm_start[0], h = sm_start[1], grp = sm_start[2];
    Seen seen = seen_of<MODE, GT>(a, b, bad);
    pdl_launch_dependents();
    // (4 bits: reported at the end, as loads behind a branch wait for it; 16 bits: no register is left for that)
    uint32_t flags = 0;
    auto report = [&](uint32_t flag) {
        if constexpr (Q4)
            flags |= flag;
        else
            atomicOr(a.status, flag);
    };

    while (at < stop) {
        // of the unit's groups those from grp on, up to `end`; the unit's begin and end in the whole batch's order
        const int end = grp + min(stop - at, seen.groups - grp);
        int u0 = at - grp, u1 = u0 + seen.groups;
        at = u0 + end;
        if (!Q4 && tid == 0) {
            sm_begin = u0;
            sm_end = u1;
            sm_done[(b * a.Hkv + h) & 1] = at;
        }
        const int32_t *set = MODE == 1 ? a.idx + ((size_t)b * a.Hkv + h) * a.top_k : nullptr;

        // Where a token of group i lies, in three steps that are taken for later groups
        // while earlier ones are computed: its position, its page, its row.  A lane
        // has token lane % GT of the group.
        auto position = [&](int i) {
            const int t = i * GT + (threadIdx.x & (GT - 1));
            if (i >= end || t >= seen.count)
                return -1;
            if (MODE == 1)
                return set[t];
            return t < seen.w.first ? t : seen.w.low + t - seen.w.first;
        };
        auto checked = [&](int p) {
            if (MODE == 1 && (p < -1 || p >= seen.n)) {
                report(kFlagIndexOutOfRange);
                return -1;
            }
            return p;
        };
        auto page = [&](int p) { return p >= 0 ? page_of(a.rows, b, p) : 0; };
        auto find = [&](int p, int pg) {
            if (p < 0)
                return -1;
            const int row = row_of(a.rows, a.Hkv, h, p, pg);
            if (row < 0)
                report(kFlagPageOutOfRange);
            return row;
        };
        Block blk[Q4 ? 1 : U];
        auto load_k = [&](int row) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int rows[2] = {__shfl_sync(kFull, row, 16 * u + r), __shfl_sync(kFull, row, 16 * u + 8 + r)};
                if constexpr (!Q4)
                    blk[u].load_k(a.rows, r, c, rows);
            }
        };
        auto load_v = [&](int row) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int at = 16 * u + 2 * c;
                const int rows[4] = {__shfl_sync(kFull, row, at), __shfl_sync(kFull, row, at + 1),
                                     __shfl_sync(kFull, row, at + 8), __shfl_sync(kFull, row, at + 9)};
                if constexpr (!Q4)
                    blk[u].load_v(a.rows, r, c, rows);
            }
        };

        // Positions, pages and rows of the warp's next groups: row is that of group i (16 bits), or
        // of the next group to fill a stage with (4 bits).
        int i = grp + warp;
        int p0 = checked(position(i)), p1 = checked(position(i + kWarps)), p2 = position(i + 2 * kWarps);
        int pg0 = page(p0), pg1 = page(p1);
        int row = find(p0, pg0), ahead = i;           // ahead: the group whose row `row` is
        auto next_row = [&] {
            p2 = checked(p2);
            const int pg2 = page(p2), p3 = position(ahead + 3 * kWarps);
            const int next = find(p1, pg1);
            p1 = p2;
            pg1 = pg2;
            p2 = p3;
            ahead += kWarps;
            return next;
        };
        uint32_t stage = ring;                        // 4 bits: the stage of group i
        auto fill = [&](uint32_t to) {                // with the rows of group `ahead`
            if constexpr (Q4) {
                if (ahead < end) {
                    Block::fill(a.rows, to, row, lane);
                    row = next_row();
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        };
        if constexpr (Q4) {
#pragma unroll 1
            for (int s = 0; s < kStages - 1; ++s)
                fill(ring + s * kStageBytes);
        } else if (i < end) {
            load_k(row);
            load_v(row);
        }

        // q of head r; a 4-bit cache's products are of fp16 values: the head's q, times a power
        // of two that brings its largest value to 2^8 (values 2^-22 times as large keep all bits)
        uint32_t q[16];
        float x2[2];             // logits to exponents of 2, heads 2c and 2c + 1
        {
            const uint16_t *src = a.q + ((size_t)b * a.Hq + (size_t)h * a.G + r) * kHeadDim;
#pragma unroll
            for (int w = 0; w < 16; w += 2) {
                const uint2 y = r < a.G ? *reinterpret_cast<const uint2 *>(src + Block::qdim(c, w)) : make_uint2(0, 0);
                q[w] = y.x;
                q[w + 1] = y.y;
            }
            x2[0] = x2[1] = MODE == 2 ? kLog2e : a.scale2;
            if constexpr (Q4) {
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < 16; ++w)
                    top = __vmaxu2(top, q[w] & 0x7fff7fffu);
                top = max(top & 0xffffu, top >> 16);
                top = max(top, __shfl_xor_sync(kFull, top, 1));
                top = max(top, __shfl_xor_sync(kFull, top, 2));
                const int e = top >> 7;                            // exponent bits of the largest
                const int up = e == 0 || e == 255 ? 0 : max(-120, min(120, 135 - e));
                const float f = __uint_as_float((uint32_t)(127 + up) << 23);
                const float inv = __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
                for (int w = 0; w < 16; ++w)
                    q[w] = pack_f16(bf_lo(q[w]) * f, bf_hi(q[w]) * f);
                x2[0] *= __shfl_sync(kFull, inv, 8 * c);
                x2[1] *= __shfl_sync(kFull, inv, 8 * c + 4);
            }
        }

        float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.0f, 0.0f};    // l: this lane's tokens
        float o[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[k][e] = 0.0f;

        for (; i < end; i += kWarps) {
            uint32_t there;
            int next = 0;
            if constexpr (Q4) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
                __syncwarp();                         // (every lane's copies; and the stage before has been read)
                fill(stage == ring ? ring + (kStages - 1) * kStageBytes : stage - kStageBytes);
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(there) : "r"(stage + kStageValid) : "memory");
            } else {
                there = __ballot_sync(kFull, row >= 0);
                next = next_row();
            }
            float s[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[u][e] = 0.0f;
                if constexpr (Q4) {
                    blk[0].load_k(stage, u, r, c);
                    blk[0].s(s[u], q);
                } else {
                    blk[u].s(s[u], q);
                }
            }
            if constexpr (!Q4)
                if (i + kWarps < end)
                    load_k(next);
            // s[u][2 t + e]: token 16 u + 8 t + r, head 2c + e; as exponents of 2 times x2
            if constexpr (MODE == 2) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int in = 16 * u + 8 * t + r, at = i * GT + in;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &x = s[u][2 * t + e];
                            x *= a.scale;
                            if (2 * c + e < a.G && at < seen.count)
                                a.logits[((size_t)b * a.Hq + (size_t)h * a.G + 2 * c + e) * a.Nmax + at] =
                                    there >> in & 1u ? x : -CUDART_INF_F;
                        }
                    }
            }
            if (there != kFull) {                     // (16 tokens: twice in the word)
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (!(there >> (16 * u + 8 * t + r) & 1u))
                            s[u][2 * t] = s[u][2 * t + 1] = -CUDART_INF_F;
            }
            // The running maximum lags until a token exceeds it by 2^8: the probabilities stay below
            // 2^8, and maxima pass between lanes and O is rescaled rarely.
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[e] = fmaxf(s[0][e], s[0][2 + e]);
                if (U == 2)
                    top[e] = fmaxf(top[e], fmaxf(s[U - 1][e], s[U - 1][2 + e]));
                top[e] *= x2[e];
            }
            if (__any_sync(kFull, top[0] > m[0] + 8.0f || top[1] > m[1] + 8.0f)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], 4));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], 8));
                    top[e] = fmaxf(top[e], __shfl_xor_sync(kFull, top[e], 16));
                    const float mn = fmaxf(m[e], top[e]);
                    const float f = safe_exp2_diff(m[e], mn);
                    m[e] = mn;
                    l[e] *= f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        o[k][e] *= f;
                        o[k][e + 2] *= f;
                    }
                }
            }
            float off[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
                off[e] = m[e] == -CUDART_INF_F ? 0.0f : -m[e];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float p[2][2];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        p[t][e] = ex2(fmaf(s[u][2 * t + e], x2[e], off[e]));
                        l[e] += p[t][e];
                    }
                if constexpr (Q4) {
                    blk[0].load_v(stage, u, r, c);
                    blk[0].pv(o, p);
                } else {
                    blk[u].pv(o, p);
                }
            }
            if constexpr (Q4) {
                stage = stage == ring + (kStages - 1) * kStageBytes ? ring : stage + kStageBytes;
            } else {
                if (i + kWarps < end)
                    load_v(next);
                row = next;
            }
        }
        if constexpr (Q4) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
        }

        // ---- the segment's result: the warps' sums joined in shared memory
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(kFull, l[e], 4);
            l[e] += __shfl_xor_sync(kFull, l[e], 8);
            l[e] += __shfl_xor_sync(kFull, l[e], 16);
            const int hd = 2 * c + e;
            if (hd < a.G) {
                if (r == 0) {
                    sm_m[warp][hd] = m[e];
                    sm_l[warp][hd] = l[e];
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<float2 *>(sm_o(warp, hd) + Block::dim(k, r)) = make_float2(o[k][e], o[k][e + 2]);
            }
        }
        __syncthreads();
        // The CTAs that share this unit's groups.
        if (!Q4) {
            u0 = sm_begin;
            u1 = sm_end;
            per = sm_per;
        }
        const int c0 = u0 / per, c1 = (u1 - 1) / per;
        const bool whole = c0 == c1;
        const int slot = 2 * blockIdx.x + (u0 > (int)blockIdx.x * per);     // (its first part or another)
        const size_t row0 = (size_t)b * a.Hq + (size_t)h * a.G;
        static_assert(kThreads == kHeadDim, "a thread per dim");
        auto weight = [](float ms, float M) { return ms == -CUDART_INF_F ? 1.0f : exp2f(ms - M); };
        for (int hd = 0; hd < a.G; ++hd) {
            float M = -CUDART_INF_F, L = 0.0f, O = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                M = fmaxf(M, sm_m[w][hd]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = weight(sm_m[w][hd], M);     // (without a maximum: zeros, or NaN)
                L += sm_l[w][hd] * f;
                O += sm_o(w, hd)[tid] * f;
            }
            if (whole) {
                a.out[(row0 + hd) * kHeadDim + tid] = f32_to_bf16_rn(L == 0.0f ? 0.0f : O / L);
                if (MODE == 2 && tid == 0) {
                    a.stat_m[row0 + hd] = M;
                    a.stat_l[row0 + hd] = L;
                }
            } else {
                a.ws->part_o[slot][hd][tid] = O;
                if (tid == 0) {
                    a.ws->part_m[slot][hd] = M;
                    a.ws->part_l[slot][hd] = L;
                }
            }
        }
        __syncthreads();
        if (!whole) {
            // The barrier orders the CTA's stores before the ticket's release; in the last
            // CTA to come the acquire and the next barrier order the loads behind the others'.
            if (tid == 0) {
                unsigned ticket;
                asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                             : "=r"(ticket)
                             : "l"(a.ws->tickets + c0)
                             : "memory");
                sm_last = ticket == (unsigned)(c1 - c0);
            }
            __syncthreads();
            if (sm_last) {
                if (tid == 0)
                    a.ws->tickets[c0] = 0;
                // CTA c0's part is its second one where the unit starts inside its range.
                const int late = (int64_t)c0 * per < u0 ? 1 : 0;
                // A warp per head; the outputs of kAhead parts are on their way at a time, the maxima
                // and sums of 32.
                for (int hd = warp; hd < a.G; hd += kWarps) {
                    float M = -CUDART_INF_F, L = 0.0f;
                    float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    constexpr int kAhead = 16;
                    for (int s0 = c0; s0 <= c1; s0 += 32) {
                        auto slot_of = [&](int s) { return 2 * s + (s == c0 ? late : 0); };
                        float m1 = -CUDART_INF_F, l1 = 0.0f;
                        if (s0 + lane <= c1) {
                            m1 = __ldcg(&a.ws->part_m[slot_of(s0 + lane)][hd]);
                            l1 = __ldcg(&a.ws->part_l[slot_of(s0 + lane)][hd]);
                        }
                        float f1 = 0.0f;
#pragma unroll 1
                        for (int h0 = 0; h0 < 32 && s0 + h0 <= c1; h0 += kAhead) {
                            float4 os[kAhead];
#pragma unroll
                            for (int k = 0; k < kAhead; ++k) {
                                os[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                if (s0 + h0 + k <= c1)
                                    os[k] = __ldcg(reinterpret_cast<const float4 *>(&a.ws->part_o[slot_of(s0 + h0 + k)][hd][4 * lane]));
                            }
                            if (h0 == 0) {
                                float mn = m1;
#pragma unroll
                                for (int d = 16; d; d >>= 1)
                                    mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, d));
                                mn = fmaxf(M, mn);
                                const float keep = weight(M, mn);
                                M = mn;
                                L *= keep;
                                O.x *= keep;
                                O.y *= keep;
                                O.z *= keep;
                                O.w *= keep;
                                f1 = weight(m1, mn);
                                float sum = l1 * f1;
#pragma unroll
                                for (int d = 16; d; d >>= 1)
                                    sum += __shfl_xor_sync(kFull, sum, d);
                                L += sum;
                            }
#pragma unroll
                            for (int k = 0; k < kAhead; ++k) {
                                const float f = __shfl_sync(kFull, f1, h0 + k);
                                O.x += os[k].x * f;
                                O.y += os[k].y * f;
                                O.z += os[k].z * f;
                                O.w += os[k].w * f;
                            }
                        }
                    }
                    uint2 y = make_uint2(0u, 0u);
                    if (L != 0.0f)
                        y = make_uint2(pack_b16(O.x / L, O.y / L), pack_b16(O.z / L, O.w / L));
                    *reinterpret_cast<uint2 *>(a.out + (row0 + hd) * kHeadDim + 4 * lane) = y;
                    if (MODE == 2 && lane == 0) {
                        a.stat_m[row0 + hd] = M;
                        a.stat_l[row0 + hd] = L;
                    }
                }
            }
        }
        // ---- the next unit
        if (!Q4) {
            at = sm_done[(b * a.Hkv + h) & 1];
            stop = sm_stop;
        }
        grp = 0;
        if (at < stop && ++h == a.Hkv) {
            h = 0;
            ++b;
            seen = seen_of<MODE, GT>(a, b, bad);
        }
    }
    if (flags)
        atomicOr(a.status, flags);
}

template <bool Q4, int MODE, int U, int CTAS>
cudaError_t launch(const CacheAttnArgs &a, int sms, cudaStream_t stream)
{
    int64_t most = 0;      // groups, if every request had the most
    {
        const int64_t count = MODE == 1 ? a.top_k : a.window > 0 && a.Nmax > a.window ? (int64_t)a.window + a.sinks : a.Nmax;
        most = (int64_t)a.B * a.Hkv * ((count + 16 * U - 1) / (16 * U) + 1);
    }
    int64_t ctas = (int64_t)sms * CTAS;
    if (ctas > most)
        ctas = most;
    if (ctas > kMaxCacheCtas)
        ctas = kMaxCacheCtas;
    constexpr size_t smem = (size_t)kWarps * (Q4 ? kStages * kStageBytes : kHeads * kHeadDim * sizeof(float));
    if (smem > 48 * 1024) {
        static std::mutex mu;
        static bool ready[64] = {false};
        int dev = 0;
        cudaError_t err = cudaGetDevice(&dev);
        if (err != cudaSuccess)
            return err;
        std::lock_guard<std::mutex> lock(mu);
        if (dev < 0 || dev >= 64 || !ready[dev]) {
            err = cudaFuncSetAttribute(cache_attention_kernel<Q4, MODE, U, CTAS>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (err != cudaSuccess)
                return err;
            if (dev >= 0 && dev < 64)
                ready[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, cache_attention_kernel<Q4, MODE, U, CTAS>, a);
}

// ---- weights: a thread per position and KV head, the logits of its G heads
constexpr int kWeightThreads = 256;
constexpr int kWeightPer = 4;

__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const WeightsArgs a, int chunks)
{
    // Lengths and sums are there when this kernel may start (the attention kernel, which does not
    // write them, lets it behind its own wait for what came before): read ahead of the wait, past L1.
    // (All behind it: 17.2 us where 3 requests of up to 2K positions take 16.2.)
    const int unit = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
    const int b = unit / a.Hkv, g = unit % a.Hkv;
    const int n = min(max(__ldcg(a.seq_lens + b), 0), a.Nmax);
    const int n0 = chunk * kWeightThreads * kWeightPer + threadIdx.x;
    const size_t row0 = (size_t)b * a.Hq + (size_t)g * a.G;
    float *w = a.weights + (size_t)unit * a.Nmax;
    float sum[kWeightPer];
#pragma unroll
    for (int k = 0; k < kWeightPer; ++k) {
        const int at = n0 + k * kWeightThreads;
        sum[k] = at < n - a.fresh ? __ldcg(w + at) : 0.0f;
    }
    pdl_wait();
    pdl_launch_dependents();
    if (n0 >= n)
        return;
    for (int hd = 0; hd < a.G; ++hd) {
        const float m = a.stat_m[row0 + hd], l = a.stat_l[row0 + hd];
        const float ref = m == -CUDART_INF_F ? 0.0f : m, inv = l == 0.0f ? 0.0f : 1.0f / l;
        const float *x = a.logits + (row0 + hd) * a.Nmax;
#pragma unroll
        for (int k = 0; k < kWeightPer; ++k) {
            const int at = n0 + k * kWeightThreads;
            if (at < n)
                sum[k] += exp2f(x[at] * kLog2e - ref) * inv;
        }
    }
#pragma unroll
    for (int k = 0; k < kWeightPer; ++k) {
        const int at = n0 + k * kWeightThreads;
        if (at < n)
            w[at] = sum[k];
    }
}

}  // namespace

cudaError_t launch_cache_attention(const CacheAttnArgs &a, int sms, cudaStream_t stream)
{
    if (a.logits)
        return launch<false, 2, 1, 3>(a, sms, stream);
    if (a.rows.scales)
        return a.idx ? launch<true, 1, 2, 4>(a, sms, stream) : launch<true, 0, 2, 4>(a, sms, stream);
    return launch<false, 0, 1, 3>(a, sms, stream);
}

cudaError_t launch_weights(const WeightsArgs &a, cudaStream_t stream)
{
    const int per = kWeightThreads * kWeightPer;
    const int chunks = (a.Nmax + per - 1) / per;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hkv * chunks));
    cfg.blockDim = dim3(kWeightThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = host_pdl();
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weights_kernel, a, chunks);
}

}  // namespace td
