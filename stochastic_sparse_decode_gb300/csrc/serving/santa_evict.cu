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
// Few rows are moved by the same CTA, many by a second kernel over all SMs: `rows` destination rows of all KV heads per CTA,
// whose sources and destinations are looked up once, then copied in 16-byte pieces.
//
// 16 sequences of 4096 to 32768 keys, 8 KV heads of 128 in bf16, 2048 keys kept of each: 74 us, of which
// the move (268 MB read and written) is at the copy rate, 41, and the longest sequence's selection the
// rest: 27 us for 32768 scores on one SM, bound by instructions (first digit 14900 cycles, listing 12300,
// placing 12100).  One sequence of 8192 keys cut to 1024: 14.4 us, a chain of dependent steps (lengths
// 1.1 us, scores and first digit 2, the other two digits 3.3, placing 1.9, then the move's lookups).
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

// The indices that (sequence b, KV head kvh) keeps, into e.kept; every thread of the CTA.
template <bool kPaged>
__device__ __forceinline__ void select_keys(const EvictParams &e, int b, int kvh, int L, long long start,
                                            unsigned char *smem) {
    const Params &p = e.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    unsigned *hist = reinterpret_cast<unsigned *>(smem), *list = hist + kBins, *cache = list + kListed;
    __shared__ unsigned warp_sum_[kSelWarps], found[2], listed;
    __shared__ int warp_n[2][kSelWarps];
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
    auto row_of = [&](int blk) {  // its first cache row, -1: a bad page (a block lies on one page)
        return blk < s1 ? int(key_row<kPaged>(p, b, start, (first + blk) * 32)) : -1;
    };
    // counts one key of a bin; a warp that agrees (many equal scores) counts once
    auto count = [&](bool in, unsigned bin) {
        const unsigned first_bin = __shfl_sync(kFull, bin, 0);
        if (__all_sync(kFull, in && bin == first_bin)) {
            if (lane == 0) atomicAdd(hist + bin, 32u);
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
        const int rows = row_of(base + lane);  // of 32 blocks, a lane each
        const int m = min(32, s1 - base);
        constexpr int kAhead = 8;
        for (int j = 0; j < m; j += kAhead) {
            float x[kAhead];
            unsigned ok = 0;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int row = __shfl_sync(kFull, rows, (j + u) & 31), key = (first + base + j + u) * 32 + lane;
                const bool in = j + u < m && key >= lo && key < hi;
                ok |= unsigned(in) << u;
                x[u] = in && row >= 0 ? load(scores + row + lane) : __uint_as_float(0x7fc00000);  // a NaN
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (j + u >= m) break;
                const unsigned v = ordered(x[u]);
                const int i = (base + j + u) * 32 + lane;
                if (i < kCached) cache[i] = v;
                count(ok >> u & 1, v >> 21);
            }
        }
    }
    find(21);
    const unsigned top = prefix;
    clear();
    // Four neighbouring keys per lane, 128 of the warp's stretch at a time, in order: f(index of the first,
    // their scores, of which of them are of the middle a bit each).  Those not held are read again.
    auto each = [&](auto f) {
        for (int i0 = s0 * 32; i0 < s1 * 32; i0 += 128) {
            const int i = i0 + 4 * lane, key = first * 32 + i;
            unsigned v[4] = {0u, 0u, 0u, 0u}, in = 0;
            if (i < s1 * 32) {
#pragma unroll
                for (int u = 0; u < 4; ++u) in |= unsigned(key + u >= lo && key + u < hi) << u;
                if (i < kCached) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(cache + i);
                    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
                } else if (in) {
                    const long long row = key_row<kPaged>(p, b, start, key);  // (keys 4 k .. 4 k + 3: on one page)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (row >= 0 && (in >> u & 1)) v[u] = ordered(load(scores + row + u));
                }
            }
            f(i, v, in);
        }
    };
    // one key per bin and lane; where a warp's 128 keys share one, once
    auto count4 = [&](const unsigned (&v)[4], unsigned in, int shift, unsigned mask) {
        const unsigned bin = v[0] >> shift & mask, first_bin = __shfl_sync(kFull, bin, 0);
        const bool same = in == 15 && bin == first_bin && (v[1] >> shift & mask) == bin && (v[2] >> shift & mask) == bin &&
                          (v[3] >> shift & mask) == bin;
        if (__all_sync(kFull, same)) {
            if (lane == 0) atomicAdd(hist + bin, 128u);
            return;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (in >> u & 1) atomicAdd(hist + (v[u] >> shift & mask), 1u);
    };
    // the keys above the bin are counted, those of the bin listed (with the warp whose stretch they are
    // of, in place of the digit that they share) and counted by the next digit
    int above = 0;
    each([&](int, const unsigned (&v)[4], unsigned in) {
        unsigned those = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            above += (in >> u & 1) && v[u] >> 21 > top >> 21;
            those |= unsigned((in >> u & 1) && v[u] >> 21 == top >> 21) << u;
        }
        if (!__any_sync(kFull, those != 0)) return;
        if (those) {
            unsigned at = atomicAdd(&listed, unsigned(__popc(those)));
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (those >> u & 1) {
                    if (at < kListed) list[at] = (v[u] & 0x1fffff) | unsigned(warp) << 21;
                    ++at;
                }
        }
        count4(v, those, 10, 2047);
    });
    find(10);
    const bool all_listed = listed <= kListed;
    const int in_list = int(min(listed, unsigned(kListed)));
    __syncthreads();
    clear();
    if (all_listed) {
        for (int i = threadIdx.x; i < in_list; i += kSelThreads)
            if ((list[i] >> 10 & 2047) == (prefix >> 10 & 2047)) atomicAdd(hist + (list[i] & 1023), 1u);
    } else {
        each([&](int, const unsigned (&v)[4], unsigned in) {
            unsigned those = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) those |= unsigned((in >> u & 1) && v[u] >> 10 == prefix >> 10) << u;
            count4(v, those, 0, 1023);
        });
    }
    find(0);
    // keys above `prefix` stay, and the first `left` of those equal to it: how many a warp's stretch has of both
    int equal = 0;
    if (!all_listed) {
        above = 0;
        each([&](int, const unsigned (&v)[4], unsigned in) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                above += (in >> u & 1) && v[u] > prefix;
                equal += (in >> u & 1) && v[u] == prefix;
            }
        });
    }
    above = __reduce_add_sync(kFull, above);
    equal = __reduce_add_sync(kFull, equal);
    if (lane == 0) {
        warp_n[0][warp] = above;
        warp_n[1][warp] = equal;
    }
    if (all_listed) {
        __syncthreads();
        for (int i = threadIdx.x; i < in_list; i += kSelThreads) {
            const unsigned v = list[i] & 0x1fffff, w = list[i] >> 21, mark = prefix & 0x1fffff;
            if (v >= mark) atomicAdd(&warp_n[v == mark][w], 1);
        }
    }
    __syncthreads();
    const bool before = lane < warp;  // the stretches before
    int na = __reduce_add_sync(kFull, before ? warp_n[0][lane] : 0), ne = __reduce_add_sync(kFull, before ? warp_n[1][lane] : 0);
    // a key that stays goes behind all above it in the order, and as many of the equal ones as stay
    each([&](int i, const unsigned (&v)[4], unsigned in) {
        int mine = 0;  // the lane's keys above (low half) and equal
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (in >> u & 1) mine += v[u] > prefix ? 1 : v[u] == prefix ? 1 << 16 : 0;
        int scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, scan, o);
            if (lane >= o) scan += x;
        }
        const int all = __shfl_sync(kFull, scan, 31);
        int a = na + ((scan - mine) & 0xffff), q = ne + ((scan - mine) >> 16);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!(in >> u & 1) || v[u] < prefix) continue;
            const bool tie = v[u] == prefix;
            // (k of them as counted; it can only be others where the scores change while this runs)
            const unsigned slot = unsigned(a + min(q, int(left)));
            if ((!tie || q < int(left)) && slot < unsigned(k)) kept[lo + slot] = first * 32 + i + u;
            a += !tie;
            q += tie;
        }
        na += all & 0xffff;
        ne += all >> 16;
    });
}

// The cache row of kept key i, -1 for a bad page id (flagged) or what is no index.
template <bool kPaged>
__device__ __forceinline__ long long row_in(const Params &p, int b, long long start, int i) {
    if (i < 0 || i >= p.max_len) return -1;
    const long long row = key_row<kPaged>(p, b, start, i);
    return row < p.total_tokens ? row : -1;
}
// Where sequence b goes: its first row, or -1 (flagged) where it does not fit; `table_out`: 0.
__device__ __forceinline__ long long first_row_out(const EvictParams &e, int b, int n) {
    if (e.table_out) return 0;
    const long long to = e.indptr_out[b], end = e.indptr_out[b + 1];
    if (to >= 0 && end <= e.rows_out && end - to >= n) return to;
    raise_flag(e.p, SANTA_ERR_INDPTR);
    return -1;
}
// The row that receives its j-th key, -1 (flagged) for a bad page id.
__device__ __forceinline__ long long row_out(const EvictParams &e, int b, long long to, int j) {
    if (!e.table_out) return to + j;
    const int pg = load(e.table_out + (size_t)b * e.max_pages_out + j / e.page_size_out);
    if (pg >= 0 && (pg + 1LL) * e.page_size_out <= e.rows_out) return (long long)pg * e.page_size_out + j % e.page_size_out;
    raise_flag(e.p, SANTA_ERR_INDPTR);
    return -1;
}

// kMove: the CTA also moves the rows of its head, 16 bytes per thread, `vecs` threads per row.
template <bool kPaged, bool kMove>
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams e, int vecs) {
    const Params &p = e.p;
    const int kvh = blockIdx.x, b = blockIdx.y;
    extern __shared__ __align__(16) unsigned char smem[];
    pdl_wait();
    pdl_launch_dependents();
    long long start;
    const int L = seq_bounds<kPaged>(p, b, &start);
    select_keys<kPaged>(e, b, kvh, L, start, smem);
    if constexpr (kMove) {
        const int n = min(L, e.keep);
        const long long to = first_row_out(e, b, n);
        if (n == 0 || to < 0) return;
        __syncthreads();  // the indices, by all threads
        const int *kept = e.kept + (size_t(b) * p.Hkv + kvh) * e.keep;
        const uint4 *k = static_cast<const uint4 *>(p.k), *v = static_cast<const uint4 *>(p.v);
        uint4 *ko = static_cast<uint4 *>(e.k_out), *vo = static_cast<uint4 *>(e.v_out);
        constexpr int kAhead = 4;
        const int vec = threadIdx.x % vecs, step = kSelThreads / vecs;
        for (int j = threadIdx.x / vecs; j < n; j += step * kAhead) {
            uint4 x[kAhead], y[kAhead];
            long long at[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                at[u] = -1;
                if (j + u * step >= n) continue;
                const long long from = row_in<kPaged>(p, b, start, kept[j + u * step]);
                at[u] = row_out(e, b, to, j + u * step);
                if (from < 0) at[u] = -1;
                if (at[u] < 0) continue;
                x[u] = load(k + (from * p.Hkv + kvh) * vecs + vec);
                y[u] = load(v + (from * p.Hkv + kvh) * vecs + vec);
                if (e.scores_out && vec == 0)
                    e.scores_out[size_t(kvh) * e.rows_out + at[u]] = load(e.scores + size_t(kvh) * p.total_tokens + from);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (at[u] >= 0) {
                    ko[(at[u] * p.Hkv + kvh) * vecs + vec] = x[u];
                    vo[(at[u] * p.Hkv + kvh) * vecs + vec] = y[u];
                }
        }
    }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveBytes = 96 * 1024;  // of K and V of a head, that its selecting CTA moves itself
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
    long long start = 0;
    if (!kPaged) start = p.kv_indptr[b];
    const long long to = first_row_out(e, b, e.lens_out[b]);
    if (to < 0) return;
    const uint4 *k = static_cast<const uint4 *>(p.k), *v = static_cast<const uint4 *>(p.v);
    uint4 *ko = static_cast<uint4 *>(e.k_out), *vo = static_cast<uint4 *>(e.v_out);
    for (int t0 = 0; t0 < n * p.Hkv; t0 += kMoveTasks) {
        const int count = min(kMoveTasks, n * p.Hkv - t0);
        __syncthreads();
        for (int t = threadIdx.x; t < count; t += kMoveThreads) {
            const int h = (t0 + t) % p.Hkv, j = j0 + (t0 + t) / p.Hkv;
            const long long from = row_in<kPaged>(p, b, start, e.kept[(size_t(b) * p.Hkv + h) * e.keep + j]);
            const long long at = row_out(e, b, to, j);
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
    const int most = e.keep < p.max_len ? e.keep : p.max_len, vecs = p.D * (dtype == SANTA_BF16 ? 2 : 4) / 16;
    // A head's CTA moves its rows itself while they are few: the second kernel costs 3 us and a launch on
    // the host, a CTA moves 512 bytes in 20 to 30 ns (8 heads of 138 rows, 70 KB each: 10.3 us with one kernel,
    // 11.0 with two; 8 heads of 300 rows, 154 KB each: 15.0 and 13.7).
    const bool move_too = (long long)most * vecs * 32 <= kMoveBytes;
    auto select = [&](auto kern) {
        const cudaError_t r = ensure_smem(kern, kSelSmem);
        return r != cudaSuccess ? r
                                : launch_kernel(kern, heads, dim3(kSelThreads), smem, stream, true, 0, false, e, vecs);
    };
    cudaError_t r;
    if (move_too)
        r = paged ? select(evict_select_kernel<true, true>) : select(evict_select_kernel<false, true>);
    else
        r = paged ? select(evict_select_kernel<true, false>) : select(evict_select_kernel<false, false>);
    if (r != cudaSuccess || most == 0 || move_too) return r;
    // as many rows per CTA as leave four CTAs per SM
    int rows = 64;
    while (rows > 1 && (long long)((most + rows - 1) / rows) * p.B < 4 * 152) rows /= 2;
    const dim3 grid(unsigned((most + rows - 1) / rows), unsigned(p.B));
    auto move = [&](auto kern) {
        return launch_kernel(kern, grid, dim3(kMoveThreads), 0, stream, true, 0, false, e, rows);
    };
    if (vecs == 8) return paged ? move(evict_move_kernel<8, true>) : move(evict_move_kernel<8, false>);
    if (vecs == 16) return paged ? move(evict_move_kernel<16, true>) : move(evict_move_kernel<16, false>);
    return paged ? move(evict_move_kernel<32, true>) : move(evict_move_kernel<32, false>);
}

}  // namespace santa
