// td_spec_api.cu -- C ABI of the speculative-decoding operators: argument
// checks, workspace layout and launches.  Every check runs on the host before
// anything is launched.
#include <cuda_runtime.h>
#include <stdint.h>

#include "td_spec.h"

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

td_status check_ws(const void *ws, size_t ws_bytes, size_t need)
{
    if (!ws || !aligned(ws, kAlign))
        return TD_ERR_INVALID_ARG;
    return ws_bytes < need ? TD_ERR_WORKSPACE_TOO_SMALL : TD_OK;
}

// The rows of a cache; `positions`: the call follows positions of requests.
td_status check_cache(const td_shape &s, const td_cache *c, bool positions)
{
    if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
        return TD_ERR_INVALID_ARG;
    if (c->num_pages < 1 || c->page_size < 1)
        return TD_ERR_INVALID_ARG;
    if ((int64_t)c->num_pages * c->page_size >= (int64_t(1) << 31) ||
        (int64_t)c->num_pages * c->page_size * s.num_kv_heads >= (int64_t(1) << 31))
        return TD_ERR_UNSUPPORTED_SHAPE;
    if (!positions)
        return TD_OK;
    if (!c->block_table)
        return c->num_pages >= s.batch && c->page_size >= s.max_seq_len ? TD_OK : TD_ERR_INVALID_ARG;
    if (!aligned(c->block_table, 4) || c->max_blocks < 1 ||
        (int64_t)c->max_blocks * c->page_size < s.max_seq_len)
        return TD_ERR_INVALID_ARG;
    return TD_OK;
}

// Workspace of the tree attention: the status word at the buffer's start, the
// rest at its end (offsets from the start of that part).
struct TreeWs {
    size_t plan, part_m, part_l, part_o, total;
};

TreeWs tree_ws(const td_shape &s, int tree_size)
{
    const size_t align = kAlign - 1;
    const size_t rows = 2 * (size_t)td::kMaxTreeCtas *
                        td::tree_part_rows(tree_size * (s.num_q_heads / s.num_kv_heads));
    TreeWs w{};
    size_t off = 0;
    w.plan = off;
    off += (td::kMaxTreeCtas * sizeof(td::JoinPlan) + align) & ~align;
    w.part_m = off;
    off += (rows * sizeof(float) + align) & ~align;
    w.part_l = off;
    off += (rows * sizeof(float) + align) & ~align;
    w.part_o = off;
    off += rows * kHeadDim * sizeof(float);
    w.total = kAlign + off;
    return w;
}

td::CacheArgs cache_args(const td_cache &c)
{
    return td::CacheArgs{(uint16_t *)c.k, (uint16_t *)c.v, c.block_table, c.num_pages, c.page_size,
                         c.max_blocks};
}

td_status run_tree(const td_shape *shape, const td_cache *cache, int32_t tree_size,
                   const int32_t *tree_lens, const uint32_t *tree_mask, const void *q,
                   const int32_t *seq_lens, const int32_t *idx, int32_t top_k, void *out, void *ws,
                   size_t ws_bytes, void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    if (tree_size < 1 || tree_size > TD_MAX_TREE)
        return TD_ERR_INVALID_ARG;
    if (shape->max_seq_len > (1 << 30))     // positions stay below 2^31 when rounded up to tiles
        return TD_ERR_UNSUPPORTED_SHAPE;
    st = check_cache(*shape, cache, true);
    if (st)
        return st;
    {   // the kernel counts its tiles of work in 31 bits
        const int64_t rows = (int64_t)tree_size * (shape->num_q_heads / shape->num_kv_heads);
        const int64_t tiles = (idx ? top_k : shape->max_seq_len) / 128 + 2;
        if ((int64_t)shape->batch * shape->num_kv_heads * ((rows + 127) / 128) * tiles > (int64_t(1) << 30))
            return TD_ERR_UNSUPPORTED_SHAPE;
    }
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !i32(seq_lens))
        return TD_ERR_INVALID_ARG;
    if ((tree_lens && !aligned(tree_lens, 4)) || (tree_mask && !aligned(tree_mask, 4)))
        return TD_ERR_INVALID_ARG;
    st = check_ws(ws, ws_bytes, td_tree_workspace_size(shape, tree_size));
    if (st)
        return st;
    td::TreeArgs a{};
    a.c = cache_args(*cache);
    a.q = (const uint16_t *)q;
    a.out = (uint16_t *)out;
    a.seq_lens = seq_lens;
    a.tree_lens = tree_lens;
    a.mask = tree_mask;
    a.idx = idx;
    a.status = (uint32_t *)ws;
    a.G = shape->num_q_heads / shape->num_kv_heads;
    a.g_shift = a.G == 1 ? 0 : a.G == 2 ? 1 : a.G == 4 ? 2 : 3;
    {
        const uint32_t d = (uint32_t)cache->page_size;
        int s = 0;
        while ((uint32_t(1) << s) < d)
            ++s;
        a.page_shift = 31 + s;
        a.page_magic = (uint32_t)(((uint64_t(1) << (31 + s)) + d - 1) / d);
    }
    a.part_rows = td::tree_part_rows(tree_size * a.G);
    const TreeWs w = tree_ws(*shape, tree_size);
    char *base = (char *)ws + (ws_bytes - (w.total - kAlign)) / kAlign * kAlign;
    a.plan = (td::JoinPlan *)(base + w.plan);
    a.part_m = (float *)(base + w.part_m);
    a.part_l = (float *)(base + w.part_l);
    a.part_o = (float *)(base + w.part_o);
    const long rows = (long)cache->num_pages * shape->num_kv_heads * cache->page_size;
    const int ps = cache->page_size;
    a.box_rows = !cache->block_table || ps % 128 == 0 ? 128 : ps >= 8 && 128 % ps == 0 ? ps : 0;
    if (!td::host_box_map(&a.box_k, cache->k, rows, a.box_rows ? a.box_rows : 1) ||
        !td::host_box_map(&a.box_v, cache->v, rows, a.box_rows ? a.box_rows : 1))
        return TD_ERR_CUDA;
    a.B = shape->batch;
    a.T = tree_size;
    a.W = (tree_size + 31) / 32;
    a.Hq = shape->num_q_heads;
    a.Hkv = shape->num_kv_heads;
    a.Nmax = shape->max_seq_len;
    a.top_k = top_k;
    a.scale = td::host_scale(*shape);
    a.wait_cycles = td::host_wait_limit_us() * 2000ll;      // of about 2 GHz
    a.wait_test = td::host_wait_test();
    return td::launch_tree_attention(a, td::host_sm_count(), (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t td_tree_workspace_size(const td_shape *shape, int32_t tree_size)
{
    if (td::host_check_shape(shape) != TD_OK || tree_size < 1 || tree_size > TD_MAX_TREE)
        return 0;
    return tree_ws(*shape, tree_size).total;
}

td_status td_tree_attn(const td_shape *shape, const td_cache *cache, int32_t tree_size,
                       const int32_t *tree_lens, const uint32_t *tree_mask, const void *q,
                       const int32_t *seq_lens, void *out, void *ws, size_t ws_bytes, void *stream)
{
    return run_tree(shape, cache, tree_size, tree_lens, tree_mask, q, seq_lens, nullptr, 0, out, ws,
                    ws_bytes, stream);
}

td_status td_tree_sparse_attn(const td_shape *shape, const td_cache *cache, int32_t tree_size,
                              const int32_t *tree_lens, const uint32_t *tree_mask, const void *q,
                              const int32_t *seq_lens, const int32_t *idx, int32_t top_k, void *out,
                              void *ws, size_t ws_bytes, void *stream)
{
    if (!i32(idx) || top_k < 1 || (shape && top_k > shape->max_seq_len))
        return TD_ERR_INVALID_ARG;
    return run_tree(shape, cache, tree_size, tree_lens, tree_mask, q, seq_lens, idx, top_k, out, ws,
                    ws_bytes, stream);
}

td_status td_tree_commit(const td_shape *shape, int32_t num_layers, const td_cache *caches,
                         int32_t tree_size, const int32_t *tree_lens, const int32_t *accepted,
                         const int32_t *accepted_lens, const int32_t *seq_lens,
                         int32_t *seq_lens_out, void *ws, size_t ws_bytes, void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    if (num_layers < 1 || !caches || tree_size < 1 || tree_size > TD_MAX_TREE)
        return TD_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l) {
        st = check_cache(*shape, &caches[l], true);
        if (st)
            return st;
        if (caches[l].num_pages != caches[0].num_pages ||
            caches[l].page_size != caches[0].page_size ||
            caches[l].max_blocks != caches[0].max_blocks ||
            caches[l].block_table != caches[0].block_table)
            return TD_ERR_INVALID_ARG;
    }
    if (!i32(accepted) || !i32(accepted_lens) || !i32(seq_lens) || !i32(seq_lens_out) ||
        (tree_lens && !aligned(tree_lens, 4)))
        return TD_ERR_INVALID_ARG;
    // other CTAs read the inputs while the new lengths are written
    const size_t bytes = (size_t)shape->batch * 4;
    if (overlap(seq_lens_out, bytes, seq_lens, bytes) ||
        overlap(seq_lens_out, bytes, tree_lens, bytes) ||
        overlap(seq_lens_out, bytes, accepted_lens, bytes) ||
        overlap(seq_lens_out, bytes, accepted, bytes * tree_size))
        return TD_ERR_INVALID_ARG;
    st = check_ws(ws, ws_bytes, kAlign);
    if (st)
        return st;
    for (int l0 = 0; l0 < num_layers; l0 += td::kAppendLayers) {
        const int nl = num_layers - l0 < td::kAppendLayers ? num_layers - l0 : td::kAppendLayers;
        td::CommitArgs a{};
        for (int j = 0; j < nl; ++j) {
            a.k[j] = (uint16_t *)caches[l0 + j].k;
            a.v[j] = (uint16_t *)caches[l0 + j].v;
        }
        a.table = caches[0].block_table;
        a.seq_lens = seq_lens;
        a.tree_lens = tree_lens;
        a.accepted = accepted;
        a.accepted_lens = accepted_lens;
        a.seq_lens_out = l0 == 0 ? seq_lens_out : nullptr;
        a.status = (uint32_t *)ws;
        a.B = shape->batch;
        a.T = tree_size;
        a.Hkv = shape->num_kv_heads;
        a.Nmax = shape->max_seq_len;
        a.num_pages = caches[0].num_pages;
        a.page_size = caches[0].page_size;
        a.max_blocks = caches[0].max_blocks;
        if (td::launch_tree_commit(a, nl, (cudaStream_t)stream) != cudaSuccess)
            return TD_ERR_CUDA;
    }
    return TD_OK;
}

td_status td_kv_append_slots(const td_shape *shape, const td_cache *cache, int32_t num_tokens,
                             const void *k_new, const void *v_new, int64_t new_stride,
                             const int32_t *slot_map, void *stream)
{
    td_status st = td::host_check_shape(shape);
    if (st)
        return st;
    st = check_cache(*shape, cache, false);
    if (st)
        return st;
    if (num_tokens < 0 || new_stride < (int64_t)shape->num_kv_heads * kHeadDim || new_stride % 8)
        return TD_ERR_INVALID_ARG;
    if (num_tokens == 0)
        return TD_OK;
    if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16) || !i32(slot_map))
        return TD_ERR_INVALID_ARG;
    td::AppendSlotsArgs a{(uint16_t *)cache->k, (uint16_t *)cache->v, (const uint16_t *)k_new,
                          (const uint16_t *)v_new, slot_map, new_stride, num_tokens,
                          shape->num_kv_heads, cache->num_pages, cache->page_size};
    return td::launch_append_slots(a, (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

td_status td_block_tables(int32_t batch, int32_t page_size, int32_t max_blocks, int32_t num_pages,
                          const int32_t *seq_lens, const int32_t *new_lens, int32_t *block_table,
                          const int32_t *num_blocks, int32_t *num_blocks_out, int32_t *free_pages,
                          const int32_t *free_count, int32_t *free_count_out, int32_t *cu_new,
                          int32_t *slot_map, int32_t max_new, void *ws, size_t ws_bytes,
                          void *stream)
{
    if (batch < 1 || page_size < 1 || max_blocks < 1 || num_pages < 1 || max_new < 0)
        return TD_ERR_INVALID_ARG;
    if (batch > 65535 || (int64_t)batch * max_blocks >= (int64_t(1) << 31) ||
        (int64_t)max_blocks * page_size >= (int64_t(1) << 31) ||
        (int64_t)num_pages * page_size >= (int64_t(1) << 31))
        return TD_ERR_UNSUPPORTED_SHAPE;
    if (!i32(seq_lens) || !i32(new_lens) || !i32(block_table) || !i32(num_blocks) ||
        !i32(num_blocks_out) || !i32(free_pages) || !i32(free_count) || !i32(free_count_out) ||
        !i32(cu_new) || (max_new > 0 && !i32(slot_map)))
        return TD_ERR_INVALID_ARG;
    td_status st = check_ws(ws, ws_bytes, kAlign);
    if (st)
        return st;
    const size_t nb = (size_t)batch * 4;
    const struct { const void *p; size_t n; } arr[] = {
        {seq_lens, nb}, {new_lens, nb}, {block_table, nb * max_blocks}, {num_blocks, nb},
        {num_blocks_out, nb}, {free_pages, (size_t)num_pages * 4}, {free_count, 4},
        {free_count_out, 4}, {cu_new, nb + 4}, {slot_map, (size_t)max_new * 4}};
    const int count = (int)(sizeof arr / sizeof arr[0]);
    for (int i = 0; i < count; ++i)
        for (int j = i + 1; j < count; ++j) {
            // in place is allowed for the two out pairs, and only exactly so
            const bool pair = (i == 3 && j == 4) || (i == 6 && j == 7);
            if (overlap(arr[i].p, arr[i].n, arr[j].p, arr[j].n) && !(pair && arr[i].p == arr[j].p))
                return TD_ERR_INVALID_ARG;
        }
    td::TablesArgs a{seq_lens, new_lens, num_blocks, free_count, block_table, num_blocks_out,
                     free_pages, free_count_out, cu_new, slot_map, (uint32_t *)ws, batch, page_size,
                     max_blocks, num_pages, max_new};
    return td::launch_block_tables(a, (cudaStream_t)stream) == cudaSuccess ? TD_OK : TD_ERR_CUDA;
}

}  // extern "C"
