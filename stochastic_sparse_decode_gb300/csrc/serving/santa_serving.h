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
    const unsigned char *kv4;  // 4-bit cache (k and v unused)
    unsigned int *cnt;         // [B][Hkv] CTAs that have stored a part of the head
    float2 *part_mz;           // [CTAs][2][G] (M, Z) of a CTA's first and last head, where others share it
    float *part;               // [CTAs][2][G][D] the unnormalised sums
};
constexpr int kSplitCtaBound = 160;  // CTAs of a split launch at most (the workspace is sized for it)
// A 3-D tensor map (santa_serving.cu); false if the driver refuses it.
bool cache_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, const cuuint64_t (&dims)[3],
               const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle);
cudaError_t launch_window(const SplitParams &p, int dtype, cudaStream_t stream, const Timing &tm);
cudaError_t launch_kv4(const SplitParams &p, int dtype, cudaStream_t stream, const Timing &tm);

}  // namespace santa
