// santa_evict.cu -- eviction by score: which keys of a (sequence, KV head) stay, and their move
// to the first rows of the sequence in another cache.
//
// Kept are the first `sinks` keys, the last `recent`, and of the n between the k = budget of
// highest score (ties: lowest index).  The k-th highest is found digit by digit (11, 11 and 10
// bits from the top) on the scores as unsigned numbers of the same order: a histogram of the
// digit, and the bin in which the count from the top passes k.  The keys of the first digit's bin
// are listed, and the other two digits look at that list alone.  No sort, and the work does not
// depend on k.  The scores lie in shared memory from the first digit on (up to kCached keys; those
// beyond are read again), the list takes up to kListed of them.
// Then every warp counts the keys of its stretch above the threshold and equal to it, one scan
// over the warps places them, and the indices are written in order.
// The move is a second kernel over all SMs: `rows` destination rows of all KV heads per CTA,
// whose sources and destinations are looked up once, then copied in 16-byte pieces.
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kSelThreads = 1024, kSelWarps = 32;
constexpr int kCached = 40960;  // scores held in shared memory
constexpr int kListed = 8192;   // keys of one bin that are listed; more are looked for among all
constexpr int kBins = 2048;
constexpr size_t kSelSmem = size_t(kCached + kListed + kBins) * 4;

// Scores as unsigned numbers of the same order; -0 is 0, a NaN 0 (below every number).
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x + 0.f);
    return x != x ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

template <bool kPaged>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams e) {
    const Params &p = e.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.x, b = blockIdx.y;
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned *hist = reinterpret_cast<unsigned *>(smem), *list = hist + kBins, *cache = list + kListed;
    __shared__ unsigned warp_sum_[kSelWarps], found[2], listed;
    __shared__ int warp_n[2][kSelWarps];
    pdl_wait();
    pdl_launch_dependents();
    long long start;
    const int L = seq_bounds<kPaged>(p, b, &start);
    const int lo = min(e.sinks, L), hi = max(lo, L - e.recent), n = hi - lo, k = min(e.budget, n);
    const int n_out = min(L, e.keep);
    if (kvh == 0 && threadIdx.x == 0) e.lens_out[b] = n_out;
    int *kept = e.kept + (size_t(b) * p.Hkv + kvh) * e.keep;
    for (int i = n_out + threadIdx.x; i < e.keep; i += kSelThreads) kept[i] = -1;
    if (k == n) {  // everything stays, or nothing of the middle where there is none
        for (int i = threadIdx.x; i < n_out; i += kSelThreads) kept[i] = i;
        return;
    }
    for (int i = threadIdx.x; i < lo; i += kSelThreads) kept[i] = i;
    for (int i = threadIdx.x; i < L - hi; i += kSelThreads) kept[lo + k + i] = hi + i;
    if (k == 0) return;
    // the blocks of 32 keys that hold the middle; a warp takes a stretch of them
    const float *scores = e.scores + size_t(kvh) * p.total_tokens;
    const int first = lo / 32, blocks = (hi + 31) / 32 - first, seg = (blocks + kSelWarps - 1) / kSelWarps;
    const int s0 = min(blocks, warp * seg), s1 = min(blocks, s0 + seg);
    auto inside = [&](int i) {  // key i of the middle's blocks
        const int key = first * 32 + i;
        return key >= lo && key < hi;
    };
    auto row_of = [&](int blk) {  // its first cache row, -1: a bad page (a block lies on one page)
        return blk < s1 ? key_row<kPaged>(p, b, start, (first + blk) * 32) : -1LL;
    };
    auto value = [&](int i) {
        if (i < kCached) return cache[i];
        if (!inside(i)) return 0u;
        const long long row = key_row<kPaged>(p, b, start, first * 32 + i);
        return row < 0 ? 0u : ordered(load(scores + row));
    };
    // counts one key of a bin; a warp that agrees (many equal scores) counts once
    auto count = [&](bool in, unsigned bin) {
        int same;
        __match_all_sync(kFull, in ? bin : 0xffffffffu, &same);
        if (same) {
            if (in && lane == 0) atomicAdd(hist + bin, 32u);
        } else if (in) {
            atomicAdd(hist + bin, 1u);
        }
    };
    auto clear = [&]() {
        for (int i = threadIdx.x; i < kBins; i += kSelThreads) hist[i] = 0;
        if (threadIdx.x == 0) listed = 0;
        __syncthreads();
    };
    unsigned prefix = 0, left = unsigned(k);  // the digits found; keys still to take among those that share them
    auto find = [&](int shift) {
        __syncthreads();
        // counts from the top: thread t holds bins 2047 - 2t and 2046 - 2t
        const unsigned h0 = hist[kBins - 1 - 2 * threadIdx.x], h1 = hist[kBins - 2 - 2 * threadIdx.x];
        unsigned s = h0 + h1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned t = __shfl_up_sync(kFull, s, o);
            if (lane >= o) s += t;
        }
        if (lane == 31) warp_sum_[warp] = s;
        __syncthreads();
        unsigned sums = warp_sum_[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned t = __shfl_up_sync(kFull, sums, o);
            if (lane >= o) sums += t;
        }
        const unsigned through = __shfl_sync(kFull, sums, warp), before = through - warp_sum_[warp] + s - h0 - h1;
        if (before < left && left <= before + h0 + h1) {  // one thread's
            const bool second = left > before + h0;
            found[0] = unsigned(kBins - 1 - 2 * threadIdx.x) - (second ? 1u : 0u);
            found[1] = left - before - (second ? h0 : 0u);
        }
        __syncthreads();
        prefix |= found[0] << shift;
        left = found[1];
    };
    clear();
    for (int base = s0; base < s1; base += 32) {
        const long long rows = row_of(base + lane);  // of 32 blocks, a lane each
        const int m = min(32, s1 - base);
        constexpr int kAhead = 8;
        for (int j = 0; j < m; j += kAhead) {
            float x[kAhead];
            bool ok[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const long long row = __shfl_sync(kFull, rows, (j + u) & 31);
                ok[u] = j + u < m && inside((base + j + u) * 32 + lane);
                x[u] = ok[u] && row >= 0 ? load(scores + row + lane) : __uint_as_float(0x7fc00000);  // a NaN
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (j + u >= m) break;
                const unsigned v = ordered(x[u]);
                const int i = (base + j + u) * 32 + lane;
                if (i < kCached) cache[i] = v;
                count(ok[u], v >> 21);
            }
        }
    }
    find(21);
    const unsigned top = prefix;
    clear();
    // the keys of the bin, listed; and counted by the next digit
    for (int i = s0 * 32 + lane; i < s1 * 32; i += 32) {
        const unsigned v = value(i);
        const bool in = inside(i) && (v & 0xffe00000u) == top;
        const unsigned those = __ballot_sync(kFull, in);
        if (!those) continue;
        unsigned at = 0;
        if (lane == 0) at = atomicAdd(&listed, unsigned(__popc(those)));
        at = __shfl_sync(kFull, at, 0) + __popc(those & ((1u << lane) - 1));
        if (in && at < kListed) list[at] = v;
        count(in, v >> 10 & 2047);
    }
    find(10);
    const bool all_listed = listed <= kListed;
    const int in_list = int(min(listed, unsigned(kListed)));
    __syncthreads();
    clear();
    if (all_listed) {
        for (int i = threadIdx.x; i < in_list; i += kSelThreads)
            if ((list[i] & 0xfffffc00u) == prefix) atomicAdd(hist + (list[i] & 1023), 1u);
    } else {
        for (int i = s0 * 32 + lane; i < s1 * 32; i += 32) {
            const unsigned v = value(i);
            count(inside(i) && (v & 0xfffffc00u) == prefix, v & 1023);
        }
    }
    find(0);
    // keys above `prefix` stay, and the first `left` of those equal to it
    int above = 0, equal = 0;
    for (int i = s0 * 32 + lane; i < s1 * 32; i += 32) {
        const unsigned v = value(i);
        const bool in = inside(i);
        above += in && v > prefix;
        equal += in && v == prefix;
    }
    above = __reduce_add_sync(kFull, above);
    equal = __reduce_add_sync(kFull, equal);
    if (lane == 0) {
        warp_n[0][warp] = above;
        warp_n[1][warp] = equal;
    }
    __syncthreads();
    const bool before = lane < warp;  // of the stretches before
    int at = __reduce_add_sync(kFull, before ? warp_n[0][lane] : 0), ties = __reduce_add_sync(kFull, before ? warp_n[1][lane] : 0);
    at += min(ties, int(left));
    const unsigned below = (1u << lane) - 1;
    for (int i = s0 * 32 + lane; i < s1 * 32; i += 32) {
        const bool in = inside(i);
        const unsigned v = value(i);
        const unsigned eq = __ballot_sync(kFull, in && v == prefix);
        const bool stays = in && (v > prefix || (v == prefix && ties + __popc(eq & below) < int(left)));
        const unsigned st = __ballot_sync(kFull, stays);
        if (stays) kept[lo + at + __popc(st & below)] = first * 32 + i;
        at += __popc(st);
        ties += __popc(eq);
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveTasks = 256;  // rows of one KV head that a CTA looks up at once

// CTA (x, y): destination rows x * rows .. + rows - 1 of sequence y, all KV heads.
template <int kVecs, bool kPaged>  // 16-byte pieces of a row
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams e, int rows) {
    const Params &p = e.p;
    const int b = blockIdx.y, j0 = blockIdx.x * rows;
    __shared__ long long src[kMoveTasks], dst[kMoveTasks];  // (row, KV head) as one number; -1: none
    pdl_wait();
    const int n = min(rows, e.lens_out[b] - j0);
    if (n <= 0) return;
    long long start = 0, to = 0;
    if (!kPaged) start = p.kv_indptr[b];
    if (!e.table_out) {
        to = e.indptr_out[b];
        const long long end = e.indptr_out[b + 1];
        if (to < 0 || end > e.rows_out || end - to < e.lens_out[b]) {
            raise_flag(p, SANTA_ERR_INDPTR);
            return;
        }
    }
    const uint4 *k = static_cast<const uint4 *>(p.k), *v = static_cast<const uint4 *>(p.v);
    uint4 *ko = static_cast<uint4 *>(e.k_out), *vo = static_cast<uint4 *>(e.v_out);
    for (int t0 = 0; t0 < n * p.Hkv; t0 += kMoveTasks) {
        const int count = min(kMoveTasks, n * p.Hkv - t0);
        __syncthreads();
        for (int t = threadIdx.x; t < count; t += kMoveThreads) {
            const int h = (t0 + t) % p.Hkv, j = j0 + (t0 + t) / p.Hkv;
            const long long from = key_row<kPaged>(p, b, start, e.kept[(size_t(b) * p.Hkv + h) * e.keep + j]);
            long long at = to + j;
            if (e.table_out) {
                const int pg = load(e.table_out + (size_t)b * e.max_pages_out + j / e.page_size_out);
                at = pg < 0 || (pg + 1LL) * e.page_size_out > e.rows_out ? -1
                                                                         : (long long)pg * e.page_size_out + j % e.page_size_out;
                if (at < 0) raise_flag(p, SANTA_ERR_INDPTR);
            }
            const bool ok = from >= 0 && at >= 0;
            src[t] = ok ? from * p.Hkv + h : -1;
            dst[t] = at * p.Hkv + h;
            if (ok && e.scores_out)
                e.scores_out[size_t(h) * e.rows_out + at] = load(e.scores + size_t(h) * p.total_tokens + from);
        }
        __syncthreads();
        constexpr int kAhead = 4, kStep = kMoveThreads / kVecs;
        const int vec = threadIdx.x % kVecs;
        for (int t = threadIdx.x / kVecs; t < count; t += kStep * kAhead) {
            uint4 a[kAhead], c[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = t + u * kStep;
                const long long s = i < count ? src[i] : -1;
                if (s >= 0) {
                    a[u] = load(k + s * kVecs + vec);
                    c[u] = load(v + s * kVecs + vec);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = t + u * kStep;
                if (i < count && src[i] >= 0) {
                    ko[dst[i] * kVecs + vec] = a[u];
                    vo[dst[i] * kVecs + vec] = c[u];
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_evict(const EvictParams &e, int dtype, cudaStream_t stream) {
    const Params &p = e.p;
    const bool paged = p.page_table != nullptr;
    const dim3 heads(unsigned(p.Hkv), unsigned(p.B));
    const int most_cached = (p.max_len + 31) / 32 * 32;  // of whole blocks
    const size_t smem = kSelSmem - (most_cached < kCached ? size_t(kCached - most_cached) * 4 : 0);
    auto select = [&](auto kern) {
        const cudaError_t r = ensure_smem(kern, kSelSmem);
        return r != cudaSuccess ? r : launch_kernel(kern, heads, dim3(kSelThreads), smem, stream, true, 0, false, e);
    };
    cudaError_t r = paged ? select(evict_select_kernel<true>) : select(evict_select_kernel<false>);
    if (r != cudaSuccess) return r;
    const int most = e.keep < p.max_len ? e.keep : p.max_len;
    if (most == 0) return cudaSuccess;
    // as many rows per CTA as leave four CTAs per SM
    int rows = 64;
    while (rows > 1 && (long long)((most + rows - 1) / rows) * p.B < 4 * 152) rows /= 2;
    const dim3 grid(unsigned((most + rows - 1) / rows), unsigned(p.B));
    auto move = [&](auto kern) {
        return launch_kernel(kern, grid, dim3(kMoveThreads), 0, stream, true, 0, false, e, rows);
    };
    const int vecs = p.D * (dtype == SANTA_BF16 ? 2 : 4) / 16;
    if (vecs == 8) return paged ? move(evict_move_kernel<8, true>) : move(evict_move_kernel<8, false>);
    if (vecs == 16) return paged ? move(evict_move_kernel<16, true>) : move(evict_move_kernel<16, false>);
    return paged ? move(evict_move_kernel<32, true>) : move(evict_move_kernel<32, false>);
}

}  // namespace santa
