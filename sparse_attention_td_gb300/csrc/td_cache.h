// td_cache.h -- kernel arguments and launchers of the operators on small caches
// (windows with sinks, 4-bit rows, attention weights and eviction), shared by
// td_cache_attn.cu, td_prompt.cu, td_cache_rows.cu and td_cache_api.cu (not part of the
// public C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/td.h"
#include "td_internal.h"
#include "td_spec.h"

namespace td {

constexpr int kCodeBytes = kHeadDim / 2;      // 4-bit codes of one K (or V) row
constexpr int kScaleBytes = kHeadDim / 8;     // scales of one token: 8 of K, 8 of V

// One layer's rows, of 16 bits ([pages][Hkv][page_size][128] bf16) or of 4 (codes
// [pages][Hkv][page_size][64] bytes, scales [..][16] bytes); table null: request b
// owns page b.
struct RowsArgs {
    const uint8_t *k, *v;
    const uint8_t *scales;      // null: rows of 16 bits
    const int32_t *table;       // [B][max_blocks]
    int num_pages, page_size, max_blocks;
    uint32_t page_magic;        // p / page_size = p * page_magic >> page_shift, 0 <= p < 2^31
    int page_shift;
};

// CTAs of a launch of the single-token kernel, at most (it sizes the partials).
constexpr int kMaxCacheCtas = 1024;

// CTAs of a launch of the kernel for many new tokens, one per SM, at most; query rows of a unit
// of its work.
constexpr int kMaxPromptCtas = 160;
constexpr int kPromptRows = 256;

// The unit that a CTA's range begins with (b -1: it has none).  rows: where the begin is the first
// cut of a unit whose tiles several CTAs share, its query rows, else 0.
struct PromptJoin {
    int b, h, q0, row0, rows, pos0;
    int last;                             // the last CTA that has a part
};

// Fixed part of the workspace, at the buffer's end whatever the shape is, so that the
// counters that have to stay zero never lie where a call of another shape writes.
struct CacheWs {
    uint32_t tickets[kMaxCacheCtas];      // parts of a cut unit that have come (zero between launches)
    float part_m[2 * kMaxCacheCtas][8];   // running maxima (log2 units)
    float part_l[2 * kMaxCacheCtas][8];   // denominators
    float part_o[2 * kMaxCacheCtas][8][kHeadDim];
    // many new tokens
    PromptJoin join[kMaxPromptCtas];
    float prompt_m[2 * kMaxPromptCtas][kPromptRows];
    float prompt_l[2 * kMaxPromptCtas][kPromptRows];
    float prompt_o[2 * kMaxPromptCtas][kPromptRows][kHeadDim];
};

// One token per request: the last one of its seq_lens[b] positions.
struct CacheAttnArgs {
    RowsArgs rows;
    const uint16_t *q;          // [B][Hq][128]
    uint16_t *out;              // [B][Hq][128]
    const int32_t *seq_lens;    // [B]
    const int32_t *idx;         // [B][Hkv][top_k], or null
    float *logits;              // weights: [B][Hq][Nmax], scaled (natural-log units); else null
    float *stat_m, *stat_l;     // weights: [B][Hq] maximum (log2 units), denominator
    uint32_t *status;
    CacheWs *ws;
    int B, Hq, Hkv, G, Nmax, top_k;
    int window, sinks;          // window 0: every position
    float scale, scale2;        // .. and times log2(e)
};
cudaError_t launch_cache_attention(const CacheAttnArgs &a, int sms, cudaStream_t stream);

// weights[b][g][n] (+)= sum over the heads h of g of softmax_h[n], from the logits
// and statistics that the attention left.
struct WeightsArgs {
    const float *logits, *stat_m, *stat_l;
    const int32_t *seq_lens;
    float *weights;             // [B][Hkv][Nmax]
    int B, Hq, Hkv, G, Nmax, fresh;
};
cudaError_t launch_weights(const WeightsArgs &a, cudaStream_t stream);

// New tokens of a packed batch: request b's are rows cu_new[b] .. cu_new[b + 1] - 1 of
// q and out, the last ones of its seq_lens[b] positions.
struct PromptArgs {
    RowsArgs rows;
    const uint16_t *q;          // [num_tokens][Hq][128]
    uint16_t *out;              // [num_tokens][Hq][128]
    const int32_t *seq_lens;    // [B]
    const int32_t *cu_new;      // [B + 1]
    uint32_t *status;
    CacheWs *ws;
    int num_tokens, B, Hq, Hkv, G, g_shift, Nmax;
    int window, sinks;          // window 0: every position
    float scale;
    long long wait_cycles;      // SM clock cycles before a wait gives up
    int wait_test;              // the softmax waits for what nothing arrives on (tests)
};
cudaError_t launch_prompt_attention(const PromptArgs &a, int sms, cudaStream_t stream);

struct Q4AppendArgs {
    uint8_t *k, *v, *scales;
    const uint16_t *k_new, *v_new;
    const int32_t *slots;
    int64_t new_stride;
    int tokens, Hkv, num_pages, page_size;
    uint32_t token_magic, page_magic;   // quotients by products (set by the launcher)
    int token_shift, page_shift;
};
cudaError_t launch_q4_append(const Q4AppendArgs &a, cudaStream_t stream);

struct EvictArgs {
    RowsArgs from, to;
    uint16_t *to_k, *to_v;
    const float *weights;       // [B][Hkv][Nmax]
    float *weights_out;         // [B][Hkv][out_row]
    const int32_t *seq_lens;
    int32_t *seq_lens_out;
    int32_t *kept;              // [B][Hkv][budget]
    uint32_t *status;
    int B, Hkv, Nmax, out_row, budget, sinks, recent;
    int place;                  // from and to are the same cache
    int pool;                   // .. or have pages of the same pool
};
cudaError_t launch_evict(const EvictArgs &a, int sms, cudaStream_t stream);

// Positions that a call sees of a request: [0, first) and [low, n).
struct Range {
    int first, low;
};
__host__ __device__ inline Range window_range(int n, int window, int sinks)
{
    const int low = window > 0 && n > window ? n - window : 0;
    return Range{sinks < low ? sinks : low, low};
}

__device__ __forceinline__ int seq_len_of(const int32_t *seq_lens, int b, int Nmax, uint32_t &bad)
{
    const int raw = seq_lens[b];
    const int n = raw < 0 ? 0 : (raw > Nmax ? Nmax : raw);
    if (n != raw)
        bad |= kFlagSeqLenOutOfRange;
    return n;
}

// Block of a request that position p >= 0 lies in: p / page_size by a product.
__device__ __forceinline__ int block_of(const RowsArgs &c, int p)
{
    return (int)((uint64_t)(uint32_t)p * c.page_magic >> c.page_shift);
}

// Page that position p of request b lies in (not yet checked).
__device__ __forceinline__ int page_of(const RowsArgs &c, int b, int p)
{
    return c.table ? c.table[(size_t)b * c.max_blocks + block_of(c, p)] : b;
}

// Cache row of position p, which lies in `page`: -1 where there is no such page.
__device__ __forceinline__ int row_of(const RowsArgs &c, int Hkv, int h, int p, int page)
{
    const int in = c.table ? p - block_of(c, p) * c.page_size : p;
    return (uint32_t)page < (uint32_t)c.num_pages ? (page * Hkv + h) * c.page_size + in : -1;
}

}  // namespace td
