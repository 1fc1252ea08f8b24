// td_spec.h -- kernel arguments, launchers and host helpers of the
// speculative-decoding operators (tree attention, commit, slot append, block
// tables), shared by td_tree.cu, td_pages.cu, td_spec_api.cu and td_api.cu
// (not part of the public C ABI).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/td.h"
#include "td_internal.h"

namespace td {

constexpr uint32_t kFlagTreeOutOfRange = 0x8u;
constexpr uint32_t kFlagPageOutOfRange = 0x10u;
constexpr uint32_t kFlagPagesExhausted = 0x20u;

// One layer's rows: k / v [num_pages][Hkv][page_size][128]; table null: request b owns page b.
struct CacheArgs {
    uint16_t *k, *v;
    const int32_t *table;    // [B][max_blocks]
    int num_pages, page_size, max_blocks;
};

// CTAs of a tree attention launch: one per SM, at most this many (it sizes the partials).
constexpr int kMaxTreeCtas = 160;

// A unit whose tiles several CTAs shared, left by the CTA whose range starts
// at the unit's first cut (rows 0: nothing to join there).
struct JoinPlan {
    int rows, b, h, row0;   // query rows of the unit, the first one's number
    int last;               // the last CTA that has a part
    int late;               // the first part is its CTA's second one
};
struct JoinArgs {
    const JoinPlan *plan;
    const float *part_m, *part_l, *part_o;
    uint16_t *out;
    int T, Hq, G, part_rows;
};

struct TreeArgs {
    TmaDesc box_k, box_v;       // rows as boxes of 64 values x box_rows rows, 128-byte swizzle
    CacheArgs c;
    const uint16_t *q;          // [B][T][Hq][128]
    uint16_t *out;              // [B][T][Hq][128]
    const int32_t *seq_lens;    // [B]
    const int32_t *tree_lens;   // [B], or null: T everywhere
    const uint32_t *mask;       // [B][T][W], or null: chain
    const int32_t *idx;         // sparse layer: [B][Hkv][top_k], or null
    uint32_t *status;
    JoinPlan *plan;             // [ctas] (written by the kernel)
    float *part_m, *part_l;     // [2 * ctas][part_rows]
    float *part_o;              // [2 * ctas][part_rows][128]
    int B, T, W, Hq, Hkv, G, Nmax, top_k;
    int g_shift;                // log2(G)
    uint32_t page_magic;        // p / page_size = p * page_magic >> page_shift, 0 <= p < 2^31
    int page_shift;
    int box_rows;               // 0: no boxes, every tile goes row by row
    int part_rows;
    float scale;                // softmax scale (natural-log units)
    long long wait_cycles;      // SM clock cycles before a wait gives up
    int wait_test;              // the softmax waits for what nothing arrives on (tests); 0 in normal use
};
// Rows one work unit of a launch with T * G query rows per KV head can have.
inline int tree_part_rows(int rows) { return rows <= 128 ? rows : 128; }
cudaError_t launch_tree_attention(const TreeArgs &a, int sms, cudaStream_t stream);

// Accepted rows of up to kAppendLayers layers in one launch.
struct CommitArgs {
    uint16_t *k[kAppendLayers];
    uint16_t *v[kAppendLayers];
    const int32_t *table;
    const int32_t *seq_lens, *tree_lens, *accepted, *accepted_lens;
    int32_t *seq_lens_out;      // null: not this launch
    uint32_t *status;
    int B, T, Hkv, Nmax, num_pages, page_size, max_blocks;
};
cudaError_t launch_tree_commit(const CommitArgs &a, int num_layers, cudaStream_t stream);

struct AppendSlotsArgs {
    uint16_t *k, *v;
    const uint16_t *k_new, *v_new;
    const int32_t *slots;
    int64_t new_stride;
    int tokens, Hkv, num_pages, page_size;
};
cudaError_t launch_append_slots(const AppendSlotsArgs &a, cudaStream_t stream);

struct TablesArgs {
    const int32_t *seq_lens, *new_lens, *held, *count;
    int32_t *table, *held_out, *free_pages, *count_out, *cu_new, *slots;
    uint32_t *status;
    int B, page_size, max_blocks, num_pages, max_new;
};
cudaError_t launch_block_tables(const TablesArgs &a, cudaStream_t stream);

// Request b's lengths as every kernel of this family reads them: seq_lens
// clamped to [0, Nmax], tree_lens to [0, min(T, n)].  `bad` collects the
// status bits of what was clamped.
struct TreeLens {
    int n;      // cached tokens, drafted ones included
    int nt;     // drafted tokens
};
__device__ __forceinline__ TreeLens tree_lens_of(const int32_t *seq_lens, const int32_t *tree_lens,
                                                 int b, int T, int Nmax, uint32_t &bad)
{
    const int raw = seq_lens[b];
    TreeLens r;
    r.n = raw < 0 ? 0 : (raw > Nmax ? Nmax : raw);
    if (r.n != raw)
        bad |= kFlagSeqLenOutOfRange;
    const int t = tree_lens ? tree_lens[b] : T;
    const int most = T < r.n ? T : r.n;
    r.nt = t < 0 ? 0 : (t > most ? most : t);
    if (r.nt != t)
        bad |= kFlagTreeOutOfRange;
    return r;
}

// Host helpers of td_api.cu.
td_status host_check_shape(const td_shape *s);
float host_scale(const td_shape &s);
int host_sm_count();
// The tuning keys "wait_limit_us" (1 s by default), "wait_test" and "pdl".
int host_wait_limit_us();
bool host_wait_test();
bool host_pdl();
// Tensor map over `rows` rows of 128 bf16 values: boxes of 64 values x box_rows
// rows, 128-byte swizzle, zero fill past the end.
bool host_box_map(TmaDesc *out, const void *base, long rows, int box_rows);

}  // namespace td
