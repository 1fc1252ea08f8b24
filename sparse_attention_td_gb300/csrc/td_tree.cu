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
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "td_attn_common.cuh"
#include "td_spec.h"

namespace td {
namespace {

constexpr int kTreeWarps = 8;

// One warp per output row; lane l holds dims 4l .. 4l + 3.
__global__ void __launch_bounds__(kTreeWarps * 32) tree_rows_kernel(const TreeArgs a)
{
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kTreeWarps + (threadIdx.x >> 5);   // t * Hq + h
    const int b = blockIdx.y;
    if (row >= a.T * a.Hq)
        return;
    const int t = row / a.Hq, h = row % a.Hq, g = h / (a.Hq / a.Hkv);
    uint32_t bad = 0;
    const TreeLens len = tree_lens_of(a.seq_lens, a.tree_lens, b, a.T, a.Nmax, bad);
    const int ctx = len.n - len.nt;
    if (bad && row == 0 && lane == 0)
        atomicOr(a.status, bad);
    if (t >= len.nt)
        return;
    const size_t at = ((size_t)b * a.T * a.Hq + row) * kHeadDim + lane * 4;
    auto load4 = [](const uint16_t *p) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
    };
    const float4 q = load4(a.q + at);
    float m = -CUDART_INF_F, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto take = [&](int p) {
        long page = b;
        int r = p;
        if (a.c.table) {
            page = a.c.table[(size_t)b * a.c.max_blocks + p / a.c.page_size];
            r = p % a.c.page_size;
            if (page < 0 || page >= a.c.num_pages) {
                if (lane == 0)
                    atomicOr(a.status, kFlagPageOutOfRange);
                return;
            }
        }
        const size_t off = (((size_t)page * a.Hkv + g) * a.c.page_size + r) * kHeadDim + lane * 4;
        const float4 k = load4(a.c.k + off);
        float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            s += __shfl_xor_sync(kFull, s, d);
        s *= a.scale * kLog2e;
        const float mn = fmaxf(m, s);
        const float keep = safe_exp2_diff(m, mn), w = exp2f(s - mn);
        const float4 v = load4(a.c.v + off);
        l = l * keep + w;
        o.x = o.x * keep + w * v.x;
        o.y = o.y * keep + w * v.y;
        o.z = o.z * keep + w * v.z;
        o.w = o.w * keep + w * v.w;
        m = mn;
    };
    if (a.idx) {
        const int32_t *ip = a.idx + ((size_t)b * a.Hkv + g) * a.top_k;
        for (int i = 0; i < a.top_k; ++i) {
            const int p = ip[i];
            if (p >= 0 && p < ctx)
                take(p);
            else if (p != -1 && lane == 0)
                atomicOr(a.status, kFlagIndexOutOfRange);
        }
    } else {
        for (int p = 0; p < ctx; ++p)
            take(p);
    }
    for (int j = 0; j < len.nt; ++j) {
        const bool sees = a.mask ? (a.mask[((size_t)b * a.T + t) * a.W + (j >> 5)] >> (j & 31)) & 1u
                                 : j <= t;
        if (sees)
            take(ctx + j);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 w;
    w.x = f32_to_bf16_rn(o.x * inv) | (uint32_t)f32_to_bf16_rn(o.y * inv) << 16;
    w.y = f32_to_bf16_rn(o.z * inv) | (uint32_t)f32_to_bf16_rn(o.w * inv) << 16;
    *reinterpret_cast<uint2 *>(a.out + at) = w;
}

}  // namespace

cudaError_t launch_tree_attention(const TreeArgs &a, cudaStream_t stream)
{
    const dim3 grid((a.T * a.Hq + kTreeWarps - 1) / kTreeWarps, a.B);
    tree_rows_kernel<<<grid, kTreeWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace td
