// td_cache_api.cu -- C ABI of the operators on small caches: argument checks, workspace
// layout and launches.  Every check runs on the host before anything is launched.
#include <cuda_runtime.h>
#include <stdint.h>

#include "td_cache.h"

namespace {

using td::kHeadDim;

constexpr size_t kAlign = 256;
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline bool i32(const void *p) { return p && aligned(p, 4); }

bool overlap(const void *a, size_t an, const void *b, size_t bn)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + bn && y < x + an;
}

// The geometry that both kinds of cache share; `positions`: rows per request that the call
// follows (0: none).
td_status check_pages(const td_shape &s, int num_pages, int page_size, const int32_t *table, int max_blocks,
                      int positions)
{
    if (num_pages < 1 || page_size < 1)
        return TD_ERR_INVALID_ARG;
    if ((int64_t)num_pages * page_size >= (int64_t(1) << 31) ||
        (int64_t)num_pages * page_size * s.num_kv_heads >= (int64_t(1) << 31))
        return TD_ERR_UNSUPPORTED_SHAPE;
    if (!positions)
        return TD_OK;
    if (!table)
        return num_pages >= s.batch && page_size >= positions ? TD_OK : TD_ERR_INVALID_ARG;
    if (!aligned(table, 4) || max_blocks < 1 || (int64_t)max_blocks * page_size < positions)
        return TD_ERR_INVALID_ARG;
    return TD_OK;
}

td_status check_rows(const td_shape &s, const td_cache *c, int positions)
{
    if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return TD_ERR_INVALID_ARG;
    return check_pages(s, c->num_pages, c->page_size, c->block_table, c->max_blocks, positions);
}

td_status check_rows(const td_shape &s, const td_q4_cache *c, int positions)
{
    if (!c || !c->k || !c->v || !c->scales || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->scales, 16))
        return TD_ERR_INVALID_ARG;
    return check_pages(s, c->num_pages, c->page_size, c->block_table, c->max_blocks, positions);
}

td::RowsArgs rows_args(const void *k, const void *v, const void *scales, const int32_t *table, int num_pages,
                       int page_size, int max_blocks)
{
    td::RowsArgs r{(const uint8_t *)k, (const uint8_t *)v, (const uint8_t *)scales, table, num_pages, page_size,
                   max_blocks, 0, 0};
    int s = 0;
    while ((uint32_t(1) << s) < (uint32_t)page_size)
        ++s;
    r.page_shift = 31 + s;
    r.page_magic = (uint32_t)(((uint64_t(1) << (31 + s)) + page_size - 1) / page_size);
    return r;
}
td::RowsArgs rows_args(const td_cache &c)
{
    return rows_args(c.k, c.v, nullptr, c.block_table, c.num_pages, c.page_size, c.max_blocks);
}
td::RowsArgs rows_args(const td_q4_cache &c)
{
    return rows_args(c.k, c.v, c.scales, c.block_table, c.num_pages, c.page_size, c.max_blocks);
}

// Workspace: the status word at the buffer's start; at its end a part of a fixed size (its
// counters have to stay zero, so they must not move with the shape), before it the softmax
// statistics of td_weights_attn.
size_t stats_bytes(const td_shape &s) { return ((size_t)s.batch * s.num_q_heads * 8 + kAlign - 1) / kAlign * kAlign; }

struct Ws {
    td::CacheWs *fixed;
    float *stat_m, *stat_l;
};

td_status cache_ws(const td_shape &s, void *ws, size_t ws_bytes, Ws &out)
{
    if (!ws || !aligned(ws, kAlign))
        return TD_ERR_INVALID_ARG;
    if (ws_bytes < td_cache_workspace_size(&s))
        return TD_ERR_WORKSPACE_TOO_SMALL;
    char *fixed = (char *)ws + (ws_bytes - sizeof(td::CacheWs)) / kAlign * kAlign;
    out.fixed = (td::CacheWs *)fixed;
    out.stat_m = (float *)(fixed - stats_bytes(s));
    out.stat_l = out.stat_m + (size_t)s.batch * s.num_q_heads;
    return TD_OK;
}

// Limits that keep a call's counts of work in 31 bits.
bool counts_fit(const td_shape &s, int64_t positions)
{
    return s.max_seq_len <= (1 << 30) &&
           (int64_t)s.batch * s.num_kv_heads * (positions / 16 + 2) <= (int64_t(1) << 30);
}

td::CacheAttnArgs token_args(const td_shape &s, const td::RowsArgs &rows, const void *q, const int32_t *seq_lens,
                             void *out, const Ws &w, void *ws)
{
    td::CacheAttnArgs a{};
    a.rows = rows;
    a.q = (const uint16_t *)q;
    a.out = (uint16_t *)out;
    a.seq_lens = seq_lens;
    a.status = (uint32_t *)ws;
    a.ws = w.fixed;
    a.B = s.batch;
    a.Hq = s.num_q_heads;
    a.Hkv = s.num_kv_heads;
    a.G = s.num_q_heads / s.num_kv_heads;
    a.Nmax = s.max_seq_len;
    a.scale = td::host_scale(s);
    a.scale2 = a.scale * 1.4426950408889634f;
    return a;
}

template <typename Cache>
td_status run_attention(const td_shape *shape, const Cache *cache, int32_t window, int32_t sinks, int32_t num_tokens,
                        const int32_t *cu_new, const void *q, const int32_t *seq_lens, void *out, void *ws,
                        size_t ws_bytes, void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    if (window < 0 || sinks < 0 || num_tokens < 0 || (!cu_new && num_tokens != shape->batch))
        return TD_ERR_INVALID_ARG;
    if (!counts_fit(*shape, shape->max_seq_len))
        return TD_ERR_UNSUPPORTED_SHAPE;
    const int G = shape->num_q_heads / shape->num_kv_heads;
    if (cu_new && ((int64_t)num_tokens * G / 256 + shape->batch) * shape->num_kv_heads > (int64_t(1) << 30))
        return TD_ERR_UNSUPPORTED_SHAPE;
    st = check_rows(*shape, cache, shape->max_seq_len);
    if (st)
        return st;
    Ws w;
    st = cache_ws(*shape, ws, ws_bytes, w);
    if (st)
        return st;
    if (!i32(seq_lens) || (cu_new && !aligned(cu_new, 4)))
        return TD_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return TD_OK;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16))
        return TD_ERR_INVALID_ARG;
    if (window >= shape->max_seq_len)
        window = 0;                        // every position
    if (sinks > shape->max_seq_len)
        sinks = shape->max_seq_len;
    if (!cu_new) {
        td::CacheAttnArgs a = token_args(*shape, rows_args(*cache), q, seq_lens, out, w, ws);
        a.window = window;
        a.sinks = sinks;
        return td::launch_cache_attention(a, td::host_sm_count(), (cudaStream_t)stream) == cudaSuccess ? TD_OK
                                                                                                      : TD_ERR_CUDA;
    }
    td::PromptArgs a{};
    a.rows = rows_args(*cache);
    a.q = (const uint16_t *)q;
    a.out = (uint16_t *)out;
    a.seq_lens = seq_lens;
    a.cu_new = cu_new;
    a.status = (uint32_t *)ws;
    a.ws = w.fixed;
    a.num_tokens = num_tokens;
    a.B = shape->batch;
    a.Hq = shape->num_q_heads;
    a.Hkv = shape->num_kv_heads;
    a.G = G;
    a.g_shift = G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3;
    a.Nmax = shape->max_seq_len;
    a.window = window;
    a.sinks = sinks;
    a.scale = td::host_scale(*shape);
    a.wait_cycles = td::host_wait_limit_us() * 2000ll;      // of about 2 GHz
    a.wait_test = td::host_wait_test();
    return td::launch_prompt_attention(a, td::host_sm_count(), (cudaStream_t)stream) == cudaSuccess ? TD_OK
                                                                                                   : TD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t td_cache_workspace_size(const td_shape *shape)
{
    if (td::host_check_shape(shape) != TD_OK)
        return 0;
    return kAlign + stats_bytes(*shape) + (sizeof(td::CacheWs) + kAlign - 1) / kAlign * kAlign;
}

td_status td_window_attn(const td_shape *shape, const td_cache *cache, int32_t window, int32_t sinks,
                         int32_t num_tokens, const int32_t *cu_new, const void *q, const int32_t *seq_lens, void *out,
                         void *ws, size_t ws_bytes, void *stream)
{
    return run_attention(shape, cache, window, sinks, num_tokens, cu_new, q, seq_lens, out, ws, ws_bytes, stream);
}

td_status td_q4_attn(const td_shape *shape, const td_q4_cache *cache, int32_t window, int32_t sinks,
                     int32_t num_tokens, const int32_t *cu_new, const void *q, const int32_t *seq_lens, void *out,
                     void *ws, size_t ws_bytes, void *stream)
{
    return run_attention(shape, cache, window, sinks, num_tokens, cu_new, q, seq_lens, out, ws, ws_bytes, stream);
}

td_status td_q4_sparse_attn(const td_shape *shape, const td_q4_cache *cache, const void *q, const int32_t *seq_lens,
                            const int32_t *idx, int32_t top_k, void *out, void *ws, size_t ws_bytes, void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    if (!i32(idx) || top_k < 1 || top_k > shape->max_seq_len)
        return TD_ERR_INVALID_ARG;
    if (!counts_fit(*shape, top_k))
        return TD_ERR_UNSUPPORTED_SHAPE;
    st = check_rows(*shape, cache, shape->max_seq_len);
    if (st)
        return st;
    Ws w;
    st = cache_ws(*shape, ws, ws_bytes, w);
    if (st)
        return st;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !i32(seq_lens))
        return TD_ERR_INVALID_ARG;
    td::CacheAttnArgs a = token_args(*shape, rows_args(*cache), q, seq_lens, out, w, ws);
    a.idx = idx;
    a.top_k = top_k;
    return td::launch_cache_attention(a, td::host_sm_count(), (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

td_status td_weights_attn(const td_shape *shape, const td_cache *cache, int32_t fresh, const void *q,
                          const int32_t *seq_lens, float *weights, float *logits, void *out, void *ws, size_t ws_bytes,
                          void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    if (fresh < 0)
        return TD_ERR_INVALID_ARG;
    if (!counts_fit(*shape, shape->max_seq_len))
        return TD_ERR_UNSUPPORTED_SHAPE;
    st = check_rows(*shape, cache, shape->max_seq_len);
    if (st)
        return st;
    Ws w;
    st = cache_ws(*shape, ws, ws_bytes, w);
    if (st)
        return st;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !i32(seq_lens) || !i32(weights) || !i32(logits))
        return TD_ERR_INVALID_ARG;
    const size_t row = (size_t)shape->max_seq_len * 4;
    if (overlap(weights, row * shape->batch * shape->num_kv_heads, logits, row * shape->batch * shape->num_q_heads))
        return TD_ERR_INVALID_ARG;
    td::CacheAttnArgs a = token_args(*shape, rows_args(*cache), q, seq_lens, out, w, ws);
    a.logits = logits;
    a.stat_m = w.stat_m;
    a.stat_l = w.stat_l;
    if (td::launch_cache_attention(a, td::host_sm_count(), (cudaStream_t)stream) != cudaSuccess)
        return TD_ERR_CUDA;
    const td::WeightsArgs x{logits, w.stat_m, w.stat_l, seq_lens, weights, a.B, a.Hq, a.Hkv, a.G, a.Nmax,
                            fresh < a.Nmax ? fresh : a.Nmax};
    return td::launch_weights(x, (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

td_status td_q4_append(const td_shape *shape, const td_q4_cache *cache, int32_t num_tokens, const void *k_new,
                       const void *v_new, int64_t new_stride, const int32_t *slot_map, void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    st = check_rows(*shape, cache, 0);
    if (st)
        return st;
    if (num_tokens < 0 || new_stride < (int64_t)shape->num_kv_heads * kHeadDim || new_stride % 8)
        return TD_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return TD_OK;
    if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16) || !i32(slot_map))
        return TD_ERR_INVALID_ARG;
    const td::Q4AppendArgs a{(uint8_t *)cache->k, (uint8_t *)cache->v, (uint8_t *)cache->scales,
                             (const uint16_t *)k_new, (const uint16_t *)v_new, slot_map, new_stride, num_tokens,
                             shape->num_kv_heads, cache->num_pages, cache->page_size, 0, 0, 0, 0};
    return td::launch_q4_append(a, (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

td_status td_evict(const td_shape *shape, const td_cache *cache, const td_cache *to, int32_t budget, int32_t sinks,
                   int32_t recent, const float *weights, float *weights_out, int32_t weights_out_row,
                   const int32_t *seq_lens, int32_t *seq_lens_out, int32_t *kept, void *ws, size_t ws_bytes,
                   void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    if (budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget)
        return TD_ERR_INVALID_ARG;
    const int64_t units = (int64_t)shape->batch * shape->num_kv_heads;
    if (shape->max_seq_len > (1 << 30) || units > (1 << 24) || units * budget >= (int64_t(1) << 40))
        return TD_ERR_UNSUPPORTED_SHAPE;
    const int most = budget < shape->max_seq_len ? budget : shape->max_seq_len;    // rows that remain
    st = check_rows(*shape, cache, shape->max_seq_len);
    if (st)
        return st;
    st = check_rows(*shape, to, most);
    if (st)
        return st;
    if (!i32(weights) || !i32(weights_out) || weights_out_row < most || !i32(seq_lens) || !i32(seq_lens_out) ||
        !i32(kept))
        return TD_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, kAlign))
        return TD_ERR_INVALID_ARG;
    if (ws_bytes < kAlign)
        return TD_ERR_WORKSPACE_TOO_SMALL;
    // The same cache (in place), pages of one pool, or two caches that share nothing.
    const size_t bytes = (size_t)cache->num_pages * cache->page_size * shape->num_kv_heads * kHeadDim * 2;
    const size_t to_bytes = (size_t)to->num_pages * to->page_size * shape->num_kv_heads * kHeadDim * 2;
    const bool pool = cache->k == to->k && cache->v == to->v && cache->num_pages == to->num_pages &&
                      cache->page_size == to->page_size;
    const bool place = pool && cache->block_table == to->block_table && cache->max_blocks == to->max_blocks;
    if (pool ? !place && (!cache->block_table || !to->block_table)
             : overlap(cache->k, bytes, to->k, to_bytes) || overlap(cache->v, bytes, to->v, to_bytes))
        return TD_ERR_INVALID_ARG;
    if (overlap(cache->k, bytes, to->v, to_bytes) || overlap(cache->v, bytes, to->k, to_bytes))
        return TD_ERR_INVALID_ARG;
    const size_t n4 = (size_t)shape->batch * 4, w4 = units * 4 * (size_t)shape->max_seq_len,
                 o4 = units * 4 * (size_t)weights_out_row, k4 = units * 4 * (size_t)budget;
    const bool same = weights == weights_out && weights_out_row == shape->max_seq_len;
    if ((!same && overlap(weights, w4, weights_out, o4)) || overlap(seq_lens, n4, seq_lens_out, n4) ||
        overlap(kept, k4, weights, w4) || overlap(kept, k4, weights_out, o4) || overlap(kept, k4, seq_lens, n4) ||
        overlap(kept, k4, seq_lens_out, n4) || overlap(seq_lens, n4, weights_out, o4) ||
        overlap(seq_lens_out, n4, weights, w4) || overlap(seq_lens_out, n4, weights_out, o4))
        return TD_ERR_INVALID_ARG;
    td::EvictArgs a{};
    a.from = rows_args(*cache);
    a.to = rows_args(*to);
    a.to_k = (uint16_t *)to->k;
    a.to_v = (uint16_t *)to->v;
    a.weights = weights;
    a.weights_out = weights_out;
    a.seq_lens = seq_lens;
    a.seq_lens_out = seq_lens_out;
    a.kept = kept;
    a.status = (uint32_t *)ws;
    a.B = shape->batch;
    a.Hkv = shape->num_kv_heads;
    a.Nmax = shape->max_seq_len;
    a.out_row = weights_out_row;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.place = place;
    a.pool = pool;
    return td::launch_evict(a, td::host_sm_count(), (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

}  // extern "C"
