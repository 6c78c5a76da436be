// santa_serving.cu -- the C entry points of the operators around the attention:
// argument checks and launches.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>

#include "santa_serving.h"

using namespace santa;

namespace {

constexpr long long kMaxRows = (1LL << 31) - 4096;  // rows of a cache: TMA row coordinates are int32

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int status(cudaError_t e) {
    if (e == cudaErrorNotSupported) return SANTA_UNSUPPORTED;
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? SANTA_OK : SANTA_CUDA_ERROR;
}
unsigned int *err_word(const santa_debug *dbg) { return dbg ? dbg->error_flags : nullptr; }

// Head layout, dtype and cache size: what every operator on heads needs.
int check_heads(const santa_problem *p) {
    if (!p) return SANTA_INVALID_ARG;
    if (p->num_q_heads < 1 || p->num_q_heads > 65535 || p->num_kv_heads < 1 || p->num_kv_heads > 65535)
        return SANTA_INVALID_ARG;
    if (p->head_dim != 64 && p->head_dim != 128) return SANTA_UNSUPPORTED;
    if (p->dtype != SANTA_F32 && p->dtype != SANTA_BF16) return SANTA_UNSUPPORTED;
    if (p->total_tokens < 0 || p->total_tokens > kMaxRows) return SANTA_INVALID_ARG;
    return SANTA_OK;
}
int check_split(const santa_problem *p) {
    const int st = check_heads(p);
    if (st != SANTA_OK) return st;
    if (p->batch < 0 || p->batch > 65535 || p->max_len < 0) return SANTA_INVALID_ARG;
    if (p->num_q_heads % p->num_kv_heads != 0) return SANTA_INVALID_ARG;
    if (p->num_q_heads / p->num_kv_heads > kMaxGroup) return SANTA_UNSUPPORTED;
    // a warp counts its blocks of 32 keys in 31 bits
    if (double(p->batch) * p->num_kv_heads * (p->max_len / 32 + 2) > 1e12) return SANTA_UNSUPPORTED;
    return SANTA_OK;
}
bool is_narrow(const santa_problem *p) {
    return p->batch <= 128 && double(p->batch) * p->num_kv_heads * (p->max_len / 32 + 2) < 2147483648.0;
}
// Rows of `heads` vectors of d elements, `stride` elements apart.
bool rows_ok(const void *base, long long stride, int heads, const santa_problem *p) {
    const int per16 = p->dtype == SANTA_BF16 ? 8 : 4;
    return aligned(base, 16) && stride >= (long long)heads * p->head_dim && stride % per16 == 0 &&
           stride <= (1LL << 40);
}

struct SplitLayout {
    size_t mz = 0, part = 0, total = 0;
};
// [B][Hkv] counters (zero between calls), then two parts per CTA of a launch.
SplitLayout split_layout(const santa_problem *p) {
    SplitLayout L;
    const size_t G = size_t(p->num_q_heads / p->num_kv_heads);
    L.mz = align256(size_t(p->batch) * p->num_kv_heads * 4);
    L.part = L.mz + align256(size_t(kSplitCtaBound) * 2 * G * sizeof(float2));
    L.total = L.part + align256(size_t(kSplitCtaBound) * 2 * G * p->head_dim * 4);
    return L;
}

// Pages of a pool of `rows` rows that hold sequences of up to max_len keys.
bool pages_ok(const santa_pages *pages, long long rows, long long max_len) {
    return pages->page_size > 0 && pages->page_size % 32 == 0 && pages->max_pages > 0 && pages->num_pages > 0 &&
           pages->num_pages <= kMaxRows / pages->page_size && pages->num_pages * pages->page_size == rows &&
           max_len <= (long long)pages->max_pages * pages->page_size;
}
bool tables_ok(const santa_pages *pages) {
    return pages->page_table && pages->kv_lens && aligned(pages->page_table, 4) && aligned(pages->kv_lens, 4);
}
// Shapes, and where the sequences lie.
Params cache_params(const santa_problem *p, const santa_pages *pages, const long long *kv_indptr, const santa_debug *dbg) {
    Params prm = {};
    prm.B = p->batch;
    prm.Hq = p->num_q_heads;
    prm.Hkv = p->num_kv_heads;
    prm.G = p->num_q_heads / p->num_kv_heads;
    prm.D = p->head_dim;
    prm.max_len = p->max_len;
    prm.total_tokens = p->total_tokens;
    prm.scale = float(1.0 / std::sqrt(double(p->head_dim)));
    prm.kv_indptr = pages ? nullptr : kv_indptr;
    if (pages) {
        prm.page_table = pages->page_table;
        prm.kv_lens = pages->kv_lens;
        prm.page_size = pages->page_size;
        prm.max_pages = pages->max_pages;
        prm.num_pages = pages->num_pages;
    }
    prm.err = err_word(dbg);
    return prm;
}
Timing timing(const santa_debug *dbg) {
    Timing tm;
    if (dbg) {
        tm.begin = reinterpret_cast<cudaEvent_t>(dbg->main_begin);
        tm.end = reinterpret_cast<cudaEvent_t>(dbg->main_end);
    }
    return tm;
}

// The attention over a cache of k and v, or, with `four_bit`, over kv4.  The keys before `first`
// do not count; own_mz (NULL: not wanted) receives each head's (M, Z): the call behind the prefix kernel.
int attend(bool four_bit, const santa_problem *p, const santa_window *w, const santa_pages *pages, const void *q,
           const void *k, const void *v, const void *kv4, const long long *kv_indptr, float *out, void *workspace,
           size_t workspace_bytes, const santa_debug *dbg, santa_stream_t stream_, int first = 0,
           float2 *own_mz = nullptr) {
    int st = check_split(p);
    if (st != SANTA_OK) return st;
    if (w && (w->window < 0 || w->sinks < 0)) return SANTA_INVALID_ARG;
    if (pages && !pages_ok(pages, p->total_tokens, p->max_len)) return SANTA_INVALID_ARG;
    if (p->batch == 0) return SANTA_OK;
    if (pages && !tables_ok(pages)) return SANTA_INVALID_ARG;
    if (!q || !out || (!kv_indptr && !pages) || !workspace) return SANTA_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || (kv_indptr && !aligned(kv_indptr, 8)))
        return SANTA_INVALID_ARG;
    const bool empty = p->max_len == 0 || p->total_tokens == 0;  // no sequence can hold a key
    const bool no_cache = four_bit ? !kv4 : !k || !v;
    if (no_cache && (!empty || k || v)) return SANTA_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv4, 16)) return SANTA_INVALID_ARG;
    const SplitLayout L = split_layout(p);
    if (workspace_bytes < L.total) return SANTA_WORKSPACE_TOO_SMALL;

    forget_error();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (empty)
        return status(cudaMemsetAsync(out, 0, size_t(p->batch) * p->num_q_heads * p->head_dim * 4, stream));

    unsigned char *ws = static_cast<unsigned char *>(workspace);
    SplitParams sp = {};
    sp.p = cache_params(p, pages, kv_indptr, dbg);
    sp.p.q = q;
    sp.p.k = k;
    sp.p.v = v;
    sp.p.out = out;
    sp.first = first;
    sp.own_mz = own_mz;
    sp.beside = own_mz != nullptr;
    sp.window = w && w->window > 0 && w->window < p->max_len ? w->window : p->max_len;
    sp.sinks = w ? w->sinks : 0;
    sp.narrow = is_narrow(p);
    sp.kv4 = static_cast<const unsigned char *>(kv4);
    sp.cnt = reinterpret_cast<unsigned int *>(ws);
    sp.part_mz = reinterpret_cast<float2 *>(ws + L.mz);
    sp.part = reinterpret_cast<float *>(ws + L.part);
    const Timing tm = timing(dbg);
    return status(four_bit ? launch_kv4(sp, p->dtype, stream, tm) : launch_window(sp, p->dtype, stream, tm));
}

struct SharedLayout {
    size_t own = 0, mz = 0, o = 0, total = 0;
};
// The own keys' workspace (whose counters come first), their (M, Z) [B][Hq], and the prefix's
// parts: a CTA begins at most one more than there are items, per stream.
SharedLayout shared_layout(const santa_problem *p) {
    SharedLayout L;
    const long long rows = (long long)p->batch * (p->num_q_heads / p->num_kv_heads);
    const size_t parts = (size_t(p->num_kv_heads) * shared_tiles(rows, p->dtype) + kSplitCtaBound) *
                         shared_streams(p->dtype) * shared_rows(p->dtype);
    L.own = split_layout(p).total;
    L.mz = L.own + align256(size_t(p->batch) * p->num_q_heads * sizeof(float2));
    L.o = L.mz + align256(parts * sizeof(float2));
    L.total = L.o + align256(parts * p->head_dim * 4);
    return L;
}

// Where pass 1 of prop leaves its records and its stash in a prop workspace (the layout stated
// at santa_decode_prop), and that workspace's size.
struct PropLayout {
    size_t rec, stash;
};
PropLayout prop_layout(const santa_problem *p) {
    PropLayout L;
    const size_t heads = size_t(p->batch) * p->num_q_heads, chunks = heads * size_t((p->max_len + 31) / 32);
    L.rec = 256 + align256(heads * 4);
    L.stash = L.rec + align256(chunks * 8) + align256(heads * 4);
    return L;
}

// Norms and rotation; `axes`: a position per axis, NULL: one per token.
int norm_rope(const santa_problem *p, const santa_rope *r, const santa_axes *axes, int num_tokens, const void *q,
              long long q_stride, const void *k, long long k_stride, const void *v, long long v_stride,
              const int *positions, const long long *slot_map, void *q_out, void *k_cache, void *v_cache,
              const santa_debug *dbg, santa_stream_t stream) {
    const int st = check_heads(p);
    if (st != SANTA_OK) return st;
    if (!r || num_tokens < 0 || num_tokens > kMaxRows) return SANTA_INVALID_ARG;
    if (r->rot_dim <= 0 || r->rot_dim > p->head_dim || r->max_pos < 1 || !(r->eps >= 0.f)) return SANTA_INVALID_ARG;
    if (r->rot_dim % 16 != 0) return SANTA_UNSUPPORTED;
    if (axes) {
        if (axes->axes < 1 || axes->axes > 4 || axes->axis_stride < num_tokens || axes->axis_stride > kMaxRows)
            return SANTA_INVALID_ARG;
        for (int i = 0; i < r->rot_dim / 2; ++i)
            if (axes->axis[i] >= axes->axes) return SANTA_INVALID_ARG;
    }
    if (num_tokens == 0) return SANTA_OK;  // before the pairs: an empty tensor has no address, its cache has one
    if (!q != !q_out || !k != !k_cache || !v != !v_cache) return SANTA_INVALID_ARG;
    if (!q && !k && !v) return SANTA_OK;
    if (!r->cos_sin || !positions || !aligned(r->cos_sin, 16) || !aligned(positions, 4) || !aligned(slot_map, 8) ||
        !aligned(r->q_weight, 16) || !aligned(r->k_weight, 16))
        return SANTA_INVALID_ARG;
    if ((q && !rows_ok(q, q_stride, p->num_q_heads, p)) || (k && !rows_ok(k, k_stride, p->num_kv_heads, p)) ||
        (v && !rows_ok(v, v_stride, p->num_kv_heads, p)) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16))
        return SANTA_INVALID_ARG;
    if (q && q == q_out && q_stride != (long long)p->num_q_heads * p->head_dim) return SANTA_INVALID_ARG;
    if (k && (k == k_cache || v == k_cache)) return SANTA_INVALID_ARG;  // rows move: not in place
    if (v && (v == v_cache || k == v_cache || k_cache == v_cache)) return SANTA_INVALID_ARG;
    forget_error();
    RopeParams rp = {};
    rp.tokens = num_tokens;
    rp.Hq = p->num_q_heads;
    rp.Hkv = p->num_kv_heads;
    rp.max_pos = r->max_pos;
    rp.rot_dim = r->rot_dim;
    rp.interleaved = r->interleaved ? 1 : 0;
    rp.eps = r->eps;
    rp.total_tokens = p->total_tokens;
    rp.q_stride = q_stride;
    rp.k_stride = k_stride;
    rp.v_stride = v_stride;
    rp.q = q;
    rp.k = k;
    rp.v = v;
    rp.q_weight = r->q_weight;
    rp.k_weight = r->k_weight;
    rp.cos_sin = r->cos_sin;
    rp.positions = positions;
    rp.slot_map = slot_map;
    rp.q_out = q_out;
    rp.k_cache = k_cache;
    rp.v_cache = v_cache;
    rp.err = err_word(dbg);
    if (axes) {
        rp.axes = axes->axes;
        rp.axis_stride = axes->axis_stride;
        for (int i = 0; i < r->rot_dim / 2; ++i) rp.axis4[i / 4] |= (unsigned char)(axes->axis[i] << 2 * (i % 4));
    }
    return status(launch_norm_rope(rp, p->dtype, p->head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

namespace santa {

bool cache_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, const cuuint64_t (&dims)[3],
               const cuuint64_t (&strides)[2], const cuuint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
    static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr)
                   : nullptr;
    }();
    const cuuint32_t step[3] = {1u, 1u, 1u};
    return encode && encode(map, type, 3, const_cast<void *>(base), dims, strides, box, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace santa

extern "C" {

int santa_page_plan(int batch, int page_size, int max_pages, long long num_pages, const int *kv_lens,
                    const int *new_lens, int *page_table, const int *free_pages, int num_free, long long *slot_map,
                    int *positions, int max_tokens, int *lens_out, int *counts, const santa_debug *dbg,
                    santa_stream_t stream) {
    if (batch < 0 || page_size < 1 || max_pages < 1 || num_pages < 0 || num_free < 0 || max_tokens < 0)
        return SANTA_INVALID_ARG;
    if (num_pages > kMaxRows / page_size || (long long)max_pages * page_size > kMaxRows ||
        max_tokens > kMaxRows)
        return SANTA_INVALID_ARG;
    if (batch > 0 && (!kv_lens || !new_lens || !page_table || !lens_out || lens_out == kv_lens || lens_out == new_lens))
        return SANTA_INVALID_ARG;
    if ((num_free > 0 && !free_pages) || (max_tokens > 0 && (!slot_map || !positions)) || !counts)
        return SANTA_INVALID_ARG;
    if (!aligned(kv_lens, 4) || !aligned(new_lens, 4) || !aligned(page_table, 4) || !aligned(free_pages, 4) ||
        !aligned(slot_map, 16) || !aligned(positions, 16) || !aligned(lens_out, 4) || !aligned(counts, 4))
        return SANTA_INVALID_ARG;
    forget_error();
    PlanParams pp = {batch,    page_size,  max_pages, num_free,  max_tokens, num_pages, kv_lens, new_lens,
                     free_pages, page_table, slot_map,  positions, lens_out,   counts,    err_word(dbg)};
    return status(launch_page_plan(pp, reinterpret_cast<cudaStream_t>(stream)));
}

int santa_norm_rope(const santa_problem *p, const santa_rope *r, int num_tokens, const void *q, long long q_stride,
                    const void *k, long long k_stride, const void *v, long long v_stride, const int *positions,
                    const long long *slot_map, void *q_out, void *k_cache, void *v_cache, const santa_debug *dbg,
                    santa_stream_t stream) {
    return norm_rope(p, r, nullptr, num_tokens, q, q_stride, k, k_stride, v, v_stride, positions, slot_map, q_out, k_cache,
                     v_cache, dbg, stream);
}

int santa_norm_rope_axes(const santa_problem *p, const santa_rope *r, const santa_axes *axes, int num_tokens,
                         const void *q, long long q_stride, const void *k, long long k_stride, const void *v,
                         long long v_stride, const int *positions, const long long *slot_map, void *q_out,
                         void *k_cache, void *v_cache, const santa_debug *dbg, santa_stream_t stream) {
    if (!axes) return SANTA_INVALID_ARG;
    return norm_rope(p, r, axes, num_tokens, q, q_stride, k, k_stride, v, v_stride, positions, slot_map, q_out, k_cache,
                     v_cache, dbg, stream);
}

int santa_kv4_size(const santa_problem *p, size_t *bytes) {
    if (!bytes) return SANTA_INVALID_ARG;
    const int st = check_heads(p);
    if (st != SANTA_OK) return st;
    *bytes = size_t(p->total_tokens) * p->num_kv_heads * kv4_record(p->head_dim);
    return SANTA_OK;
}

int santa_kv4_append(const santa_problem *p, int num_tokens, const void *k, long long k_stride, const void *v,
                     long long v_stride, const long long *slot_map, void *kv4, const santa_debug *dbg,
                     santa_stream_t stream) {
    const int st = check_heads(p);
    if (st != SANTA_OK) return st;
    if (num_tokens < 0 || num_tokens > kMaxRows) return SANTA_INVALID_ARG;
    if (num_tokens == 0) return SANTA_OK;
    if (!k || !v || !kv4 || !aligned(kv4, 16) || !aligned(slot_map, 8) || !rows_ok(k, k_stride, p->num_kv_heads, p) ||
        !rows_ok(v, v_stride, p->num_kv_heads, p))
        return SANTA_INVALID_ARG;
    forget_error();
    StoreParams sp = {};
    sp.tokens = num_tokens;
    sp.Hkv = p->num_kv_heads;
    sp.total_tokens = p->total_tokens;
    sp.k_stride = k_stride;
    sp.v_stride = v_stride;
    sp.k = k;
    sp.v = v;
    sp.slot_map = slot_map;
    sp.kv4 = static_cast<unsigned char *>(kv4);
    sp.err = err_word(dbg);
    return status(launch_kv4_append(sp, p->dtype, p->head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

int santa_kv4_read(const santa_problem *p, int num_tokens, const void *kv4, const long long *slot_map, void *k,
                   void *v, const santa_debug *dbg, santa_stream_t stream) {
    const int st = check_heads(p);
    if (st != SANTA_OK) return st;
    if (num_tokens < 0 || num_tokens > kMaxRows) return SANTA_INVALID_ARG;
    if (num_tokens == 0 || (!k && !v)) return SANTA_OK;
    if (!kv4 || !aligned(kv4, 16) || !aligned(slot_map, 8) || !aligned(k, 16) || !aligned(v, 16) || k == v ||
        k == kv4 || v == kv4)
        return SANTA_INVALID_ARG;
    forget_error();
    StoreParams sp = {};
    sp.tokens = num_tokens;
    sp.Hkv = p->num_kv_heads;
    sp.total_tokens = p->total_tokens;
    sp.slot_map = slot_map;
    sp.kv4 = static_cast<unsigned char *>(const_cast<void *>(kv4));
    sp.k_out = k;
    sp.v_out = v;
    sp.err = err_word(dbg);
    return status(launch_kv4_read(sp, p->dtype, p->head_dim, reinterpret_cast<cudaStream_t>(stream)));
}

int santa_split_workspace_size(const santa_problem *p, size_t *bytes) {
    if (!bytes) return SANTA_INVALID_ARG;
    const int st = check_split(p);
    if (st != SANTA_OK) return st;
    *bytes = split_layout(p).total;
    return SANTA_OK;
}

int santa_split_workspace_init(const santa_problem *p, void *workspace, size_t workspace_bytes,
                               santa_stream_t stream) {
    const int st = check_split(p);
    if (st != SANTA_OK) return st;
    if (!workspace || !aligned(workspace, 256)) return SANTA_INVALID_ARG;
    const SplitLayout L = split_layout(p);
    if (workspace_bytes < L.total) return SANTA_WORKSPACE_TOO_SMALL;
    forget_error();
    return status(cudaMemsetAsync(workspace, 0, L.mz, reinterpret_cast<cudaStream_t>(stream)));
}

int santa_decode_window(const santa_problem *p, const santa_window *w, const santa_pages *pages, const void *q,
                        const void *k, const void *v, const long long *kv_indptr, float *out, void *workspace,
                        size_t workspace_bytes, const santa_debug *dbg, santa_stream_t stream) {
    if (!w) return SANTA_INVALID_ARG;
    return attend(false, p, w, pages, q, k, v, nullptr, kv_indptr, out, workspace, workspace_bytes, dbg, stream);
}

int santa_decode_kv4(const santa_problem *p, const santa_window *w, const santa_pages *pages, const void *q,
                     const void *kv4, const long long *kv_indptr, float *out, void *workspace,
                     size_t workspace_bytes, const santa_debug *dbg, santa_stream_t stream) {
    return attend(true, p, w, pages, q, nullptr, nullptr, kv4, kv_indptr, out, workspace, workspace_bytes, dbg, stream);
}

int santa_shared_workspace_size(const santa_problem *p, size_t *bytes) {
    if (!bytes) return SANTA_INVALID_ARG;
    const int st = check_split(p);
    if (st != SANTA_OK) return st;
    *bytes = shared_layout(p).total;
    return SANTA_OK;
}

int santa_decode_shared(const santa_problem *p, const santa_prefix *prefix, const santa_pages *pages, const void *q,
                        const void *k, const void *v, const long long *kv_indptr, float *out, void *workspace,
                        size_t workspace_bytes, const santa_debug *dbg, santa_stream_t stream_) {
    const int st = check_split(p);
    if (st != SANTA_OK) return st;
    if (!prefix || prefix->len < 0) return SANTA_INVALID_ARG;
    if (pages) {
        if (!pages_ok(pages, p->total_tokens, p->max_len) || prefix->len > p->max_len) return SANTA_INVALID_ARG;
    } else if (prefix->start < 0 || prefix->start > p->total_tokens - prefix->len) {
        return SANTA_INVALID_ARG;
    }
    if (p->batch == 0) return SANTA_OK;
    if (pages && !tables_ok(pages)) return SANTA_INVALID_ARG;
    if (!q || !out || (!kv_indptr && !pages) || !workspace) return SANTA_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) || !aligned(k, 16) || !aligned(v, 16) ||
        (kv_indptr && !aligned(kv_indptr, 8)) || ((!k || !v) && (p->total_tokens > 0 || k || v)))
        return SANTA_INVALID_ARG;
    const SharedLayout L = shared_layout(p);
    if (workspace_bytes < L.total) return SANTA_WORKSPACE_TOO_SMALL;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    float2 *own_mz = reinterpret_cast<float2 *>(ws + L.own);
    const santa_window all = {0, 0};
    if (prefix->len == 0)  // only own keys
        return attend(false, p, &all, pages, q, k, v, nullptr, kv_indptr, out, workspace, workspace_bytes, dbg, stream_);

    forget_error();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    SharedParams sp = {};
    sp.p = cache_params(p, pages, kv_indptr, dbg);
    sp.p.q = q;
    sp.p.k = k;
    sp.p.v = v;
    sp.p.out = out;
    sp.len = prefix->len;
    sp.start = prefix->start;
    sp.rows = p->batch * sp.p.G;
    sp.tiles = shared_tiles(sp.rows, p->dtype);
    sp.nb = int(((long long)prefix->len + shared_block(p->dtype) - 1) / shared_block(p->dtype));
    sp.mz = reinterpret_cast<float2 *>(ws + L.mz);
    sp.o = reinterpret_cast<float *>(ws + L.o);
    cudaError_t e = launch_shared(sp, p->dtype, stream, timing(dbg));
    if (e != cudaSuccess) return status(e);
    const bool own = p->max_len > (pages ? prefix->len : 0);  // some sequence may have keys of its own
    if (own) {
        santa_debug d = {};
        d.error_flags = err_word(dbg);
        const int r = attend(false, p, &all, pages, q, k, v, nullptr, kv_indptr, out, workspace, L.own, &d, stream_,
                             pages ? prefix->len : 0, own_mz);
        if (r != SANTA_OK) return r;
        sp.own_mz = own_mz;
    }
    return status(launch_shared_join(sp, p->dtype, stream));
}

int santa_key_weights(const santa_problem *p, const santa_pages *pages, const void *q, const void *k,
                      const long long *kv_indptr, const float *scores, float *scores_out, float decay, int fresh,
                      void *workspace, size_t workspace_bytes, const santa_debug *dbg, santa_stream_t stream_) {
    size_t need = 0;
    const int st = santa_workspace_size(p, SANTA_MODE_PROP, &need);
    if (st != SANTA_OK) return st;
    if (pages && !pages_ok(pages, p->total_tokens, p->max_len)) return SANTA_INVALID_ARG;
    if (!(decay >= 0.f) || std::isinf(decay) || fresh < 0 || !q != !k || (pages && !q)) return SANTA_INVALID_ARG;
    if (p->batch == 0 || p->max_len == 0 || p->total_tokens == 0) return SANTA_OK;  // no key
    if (pages && !tables_ok(pages)) return SANTA_INVALID_ARG;
    if (!scores_out || !workspace || (!kv_indptr && !pages)) return SANTA_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(kv_indptr, 8) || !aligned(scores, 4) || !aligned(scores_out, 4) ||
        !aligned(workspace, 256))
        return SANTA_INVALID_ARG;
    if (workspace_bytes < need) return SANTA_WORKSPACE_TOO_SMALL;
    forget_error();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    const PropLayout L = prop_layout(p);
    WeightParams w = {};
    w.p = cache_params(p, pages, kv_indptr, dbg);
    w.p.nch = (p->max_len + 31) / 32;
    w.p.nch4 = (w.p.nch + 3) & ~3;
    w.p.tile = p->tile;
    w.p.S = 1;
    w.p.q = q;
    w.p.k = k;
    w.p.rec = reinterpret_cast<unsigned long long *>(ws + L.rec);
    w.p.stash = reinterpret_cast<float *>(ws + L.stash);
    if (q) {
        CUtensorMap map;
        const int es = p->dtype == SANTA_BF16 ? 2 : 4;
        const cuuint64_t dims[3] = {cuuint64_t(p->head_dim), cuuint64_t(p->num_kv_heads), cuuint64_t(p->total_tokens)};
        const cuuint64_t strides[2] = {cuuint64_t(p->head_dim) * es, cuuint64_t(p->num_kv_heads) * p->head_dim * es};
        const cuuint32_t box[3] = {cuuint32_t(128 / es), 1u, 32u};
        if (!cache_map(&map, p->dtype == SANTA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, k,
                       dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return SANTA_CUDA_ERROR;
        // One sequence fills prop's walk, and is 1.7 us ahead without a plan; of a batch the host does not
        // know the lengths (16 of 4096 to 32768 keys: 134 us by prop's walk, 110 by equal shares).
        cudaError_t e;
        if (p->dtype == SANTA_BF16 && p->batch > 1) {
            SplitParams sp = {};
            sp.p = w.p;
            sp.window = p->max_len;
            sp.no_join = 1;
            sp.narrow = is_narrow(p);
            e = launch_key_logits(sp, map, stream, timing(dbg));
        } else {
            e = launch_prop(w.p, p->dtype, map, stream, timing(dbg), kPass1);
        }
        if (e != cudaSuccess) return status(e);
    }
    w.scores = scores;
    w.scores_out = scores_out;
    w.decay = decay;
    w.fresh = fresh;
    return status(launch_key_weights(w, stream));
}

int santa_evict(const santa_problem *p, const santa_keep *keep, const santa_pages *pages, const void *k, const void *v,
                const float *scores, const long long *kv_indptr, void *k_out, void *v_out, float *scores_out,
                long long rows_out, const long long *indptr_out, const santa_pages *pages_out, int *kept,
                int *lens_out, const santa_debug *dbg, santa_stream_t stream) {
    const int st = check_heads(p);
    if (st != SANTA_OK) return st;
    if (p->batch < 0 || p->batch > 65535 || p->max_len < 0) return SANTA_INVALID_ARG;
    if (!keep || keep->sinks < 0 || keep->recent < 0 || keep->budget < 0) return SANTA_INVALID_ARG;
    const long long sum = (long long)keep->sinks + keep->recent + keep->budget;
    if (sum > kMaxRows || rows_out < 0 || rows_out > kMaxRows) return SANTA_INVALID_ARG;
    if (pages && !pages_ok(pages, p->total_tokens, p->max_len)) return SANTA_INVALID_ARG;
    if (pages_out && !pages_ok(pages_out, rows_out, sum < p->max_len ? sum : p->max_len)) return SANTA_INVALID_ARG;
    if (p->batch == 0) return SANTA_OK;
    if (pages && !tables_ok(pages)) return SANTA_INVALID_ARG;
    if ((pages_out && (!pages_out->page_table || !aligned(pages_out->page_table, 4))) || (!pages_out && !indptr_out) ||
        (!pages && !kv_indptr) || !lens_out || (sum > 0 && !kept))
        return SANTA_INVALID_ARG;
    const bool empty = p->max_len == 0 || p->total_tokens == 0;
    if (!empty && (!k || !v || !scores)) return SANTA_INVALID_ARG;
    if (!empty && sum > 0 && (!k_out || !v_out || k_out == v_out || k_out == v || v_out == k)) return SANTA_INVALID_ARG;
    if ((scores_out && scores_out == scores) || (pages && pages->kv_lens == lens_out)) return SANTA_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(scores, 4) ||
        !aligned(scores_out, 4) || !aligned(kv_indptr, 8) || !aligned(indptr_out, 8) || !aligned(kept, 4) ||
        !aligned(lens_out, 4))
        return SANTA_INVALID_ARG;
    forget_error();
    EvictParams e = {};
    e.p = cache_params(p, pages, kv_indptr, dbg);
    e.p.k = k;
    e.p.v = v;
    e.scores = scores;
    e.scores_out = scores_out;
    e.k_out = k_out;
    e.v_out = v_out;
    e.sinks = keep->sinks;
    e.recent = keep->recent;
    e.budget = keep->budget;
    e.keep = int(sum);
    e.rows_out = rows_out;
    e.indptr_out = pages_out ? nullptr : indptr_out;
    if (pages_out) {
        e.table_out = pages_out->page_table;
        e.page_size_out = pages_out->page_size;
        e.max_pages_out = pages_out->max_pages;
    }
    e.kept = kept;
    e.lens_out = lens_out;
    return status(launch_evict(e, p->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
