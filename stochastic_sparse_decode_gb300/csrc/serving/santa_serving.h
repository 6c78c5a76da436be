// santa_serving.h -- parameter blocks and launchers of the operators around the
// attention (page plan, norm + rotation, 4-bit cache, windowed / 4-bit attention).
#pragma once

#include "santa_launch.h"

namespace santa {

constexpr int kMaxGroup = 8;  // query heads of one KV head, at most

struct PlanParams {
    int batch, page_size, max_pages, num_free, max_tokens;
    long long num_pages;
    const int *kv_lens, *new_lens, *free_pages;
    int *page_table;
    long long *slot_map;
    int *positions, *lens_out, *counts;
    unsigned int *err;
    unsigned magic, shift;  // division by page_size (set by the launcher)
};
cudaError_t launch_page_plan(const PlanParams &p, cudaStream_t stream);

struct RopeParams {
    int tokens, Hq, Hkv, max_pos, rot_dim, interleaved;
    float eps;
    long long total_tokens, q_stride, k_stride, v_stride;
    const void *q, *k, *v, *q_weight, *k_weight;
    const float *cos_sin;
    const int *positions;
    const long long *slot_map;
    void *q_out, *k_cache, *v_cache;
    unsigned int *err;
    int axes;                   // 0: one position per token, else a position per axis
    long long axis_stride;
    unsigned char axis4[16];    // the axes of pairs 4 l .. 4 l + 3, two bits each
};
cudaError_t launch_norm_rope(const RopeParams &p, int dtype, int d, cudaStream_t stream);

struct StoreParams {
    int tokens, Hkv;
    long long total_tokens, k_stride, v_stride;
    const void *k, *v;
    const long long *slot_map;
    unsigned char *kv4;        // append: written; read: read
    void *k_out, *v_out;       // read
    unsigned int *err;
};
cudaError_t launch_kv4_append(const StoreParams &p, int dtype, int d, cudaStream_t stream);
cudaError_t launch_kv4_read(const StoreParams &p, int dtype, int d, cudaStream_t stream);

// Bytes of one 4-bit record (K and V of one token and KV head).
constexpr int kv4_record(int d) { return d + d / 8; }

// Attention over the visible keys of each sequence.  `p` carries the shapes, q, k, v,
// the cache's addressing, out and the error word as for the other modes.
struct SplitParams {
    Params p;
    int window, sinks;         // window >= max_len: every key is visible
    int narrow;                // at most 128 sequences whose units of 32 keys number below 2^31
    int first;                 // the first key that counts (a prefix before it is another kernel's)
    float2 *own_mz;            // [B][Hq] the (M, Z) that out is divided by, or NULL
    int beside;                // the kernel before is the same call's and runs beside this one (santa_window.cu)
    int no_join;               // the units' results stand alone: equal stretches, whatever the heads
    const unsigned char *kv4;  // 4-bit cache (k and v unused)
    unsigned int *cnt;         // [B][Hkv] CTAs that have stored a part of the head
    float2 *part_mz;           // [CTAs][2][G] (M, Z) of a CTA's first and last head, where others share it
    float *part;               // [CTAs][2][G][D] the unnormalised sums
};
constexpr int kSplitCtaBound = 160;  // CTAs of a split launch at most (the workspace is sized for it)
// A 3-D tensor map (santa_serving.cu); false if the driver refuses it.
bool cache_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, const cuuint64_t (&dims)[3],
               const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle);
// Attention of the batch's queries over a prefix that all sequences share, into parts, and the
// join of these with the sequences' own attention (santa_shared.cu).
struct SharedParams {
    Params p;                  // shapes, q, out, the cache's addressing (page table: sequence 0's row)
    int len;                   // keys of the prefix
    long long start;           // its first row (contiguous)
    int rows, tiles, nb;       // query rows of a KV head, tiles of them, blocks of keys
    int ctas, both;            // CTAs; both: the CTA's two streams share the blocks of one tile of rows
    float2 *mz;                // [items + CTAs][streams][tile rows] (M, Z)
    float *o;                  // [items + CTAs][streams][tile rows][D] unnormalised sums
    const float2 *own_mz;      // [B][Hq] (M, Z) of the own keys; out holds their normalised sums
};
// Streams per CTA and query rows per stream of the prefix kernel (bf16: tensor cores).
constexpr int shared_streams(int dtype) { return dtype == SANTA_BF16 ? 2 : 1; }
constexpr int shared_rows(int dtype) { return dtype == SANTA_BF16 ? 128 : 64; }
constexpr int shared_block(int dtype) { return dtype == SANTA_BF16 ? 64 : 32; }
// Tiles of the rows of one KV head: a tile fills every stream of a CTA.
inline int shared_tiles(long long rows, int dtype) {
    const int r = shared_rows(dtype) * shared_streams(dtype);
    return int((rows + r - 1) / r);
}
cudaError_t launch_shared(SharedParams &sp, int dtype, cudaStream_t stream, const Timing &tm);  // sets sp.ctas
cudaError_t launch_shared_join(const SharedParams &sp, int dtype, cudaStream_t stream);

struct WeightParams {
    Params p;                  // shapes, the cache's addressing, pass 1's records and stash
    const float *scores;
    float *scores_out;
    float decay;
    int fresh;
};
cudaError_t launch_key_weights(const WeightParams &w, cudaStream_t stream);
// Pass 1 of prop on bf16 keys, bit for bit, by equal shares of the blocks that the sequences hold.
cudaError_t launch_key_logits(const SplitParams &sp, const CUtensorMap &kmap, cudaStream_t stream, const Timing &tm);

struct EvictParams {
    Params p;                  // shapes, k, v, the cache's addressing
    const float *scores;
    float *scores_out;
    void *k_out, *v_out;
    int sinks, recent, budget, keep;  // keep: their sum
    long long rows_out;
    const long long *indptr_out;
    const int *table_out;      // NULL: contiguous
    int page_size_out, max_pages_out;
    int *kept, *lens_out;
};
cudaError_t launch_evict(const EvictParams &e, int dtype, cudaStream_t stream);

cudaError_t launch_window(const SplitParams &p, int dtype, cudaStream_t stream, const Timing &tm);
cudaError_t launch_kv4(const SplitParams &p, int dtype, cudaStream_t stream, const Timing &tm);

}  // namespace santa
