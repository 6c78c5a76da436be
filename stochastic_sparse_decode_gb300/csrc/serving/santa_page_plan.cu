// santa_page_plan.cu -- block tables and slot maps from request lengths, in one kernel.
//
// With have_b = ceil(len_b / ps), need_b = ceil((len_b + new_b) / ps) - have_b and the
// prefix sums P_b = sum_{b' < b} need_b', T_b = sum_{b' < b} max(new_b', 0):
//   page_table[b][have_b + i] = free_pages[P_b + i],                  i < need_b
//   slot_map[T_b + i] = page(b, n / ps) ps + n mod ps,  n = len_b + i,  i < new_b.
// Every CTA scans the sequences itself, kPlanThreads at a time (two block scans: the
// token counts, which decide who fits, then the page counts of those that do), so no
// CTA waits for another and one launch does it all; the CTAs then share the tile's new
// pages and tokens, found by binary searches in the tile's prefix sums: four consecutive
// tokens per thread and search, written by 16-byte stores, with the page of a position by
// multiplication (the divisor is the call's).  A page
// that a token lies in is read from the free list itself when it is new, so the table
// entries that another CTA writes are never read.
//
// Bound by latency: lengths, two scans and a search precede the first store.  64 sequences of
// one token each 4.1 us; 200 prompts of 4096 tokens on average (9.8 MB written, 1.5 us at the
// copy rate) 8.3 us, 12.5 with a search and scalar stores per token.  The prompts' 4.0 million
// warp instructions are 3.2 us of every scheduler's time, by under 4 warps each that issue in 0.42 of
// the cycles: the part behind the scans is instructions as much as it is latency.
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanCtas = 304;  // two per SM (820k tokens: 152 13.0 us, 304 8.3, 608 10.6, 912 8.4)

__device__ __forceinline__ void plan_flag(const PlanParams &p, unsigned bit) {
    if (p.err) atomicOr(p.err, bit);
}

// Inclusive scan over the block; every thread also receives the total.
__device__ __forceinline__ long long block_scan(long long v, long long *scr, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(kFull, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();  // scr may still be read from the scan before
    if (lane == 31) scr[warp] = v;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        const long long s = scr[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return v + before;
}

// First i in [0, n) with end[i] > x (n if there is none).
__device__ __forceinline__ int upper(const long long *end, int n, long long x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (end[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// pos / page_size, by the magic number of the launch: floor(pos (2^s / d rounded up) / 2^s) with
// s = 31 + ceil(log2 d) is the quotient for every 0 <= pos < 2^31.
__device__ __forceinline__ int page_of(int pos, const PlanParams &p) {
    return p.page_size == 1 ? pos : int(__umulhi(unsigned(pos), p.magic) >> p.shift);
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p) {
    __shared__ long long scr[kPlanThreads / 32];
    __shared__ long long s_tok[kPlanThreads], s_page[kPlanThreads];  // inclusive prefix sums of the tile
    __shared__ int s_len[kPlanThreads], s_have[kPlanThreads];
    __shared__ int s_ok[kPlanThreads];
    __shared__ unsigned s_sum[2];  // pages taken, tokens placed (first CTA); both below 2^31
    const int tid = threadIdx.x;
    const long long me = (long long)blockIdx.x * kPlanThreads + tid, all = (long long)gridDim.x * kPlanThreads;
    pdl_wait();
    pdl_launch_dependents();
    long long tok0 = 0, page0 = 0;  // of the tiles before
    if (tid < 2) s_sum[tid] = 0;
    __syncthreads();
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int len = 0, nw = 0;
        if (b < p.batch) {
            len = p.kv_lens[b];
            nw = p.new_lens[b];
        }
        const bool negative = len < 0 || nw < 0;
        const long long n_tok = nw > 0 ? nw : 0;
        long long tile_tok, tile_page;
        const long long tok_end = block_scan(n_tok, scr, &tile_tok);
        const long long want = ((long long)len + nw + p.page_size - 1) / p.page_size;
        bool ok = !negative && want <= p.max_pages && (n_tok == 0 || tok0 + tok_end <= p.max_tokens);
        const int have = negative ? 0 : int(((long long)len + p.page_size - 1) / p.page_size);
        const long long need = ok ? want - have : 0;
        const long long page_end = block_scan(need, scr, &tile_page);
        if (need > 0 && page0 + page_end > p.num_free) ok = false;
        s_tok[tid] = tok_end;
        s_page[tid] = page_end;
        s_len[tid] = len;
        s_have[tid] = have;
        s_ok[tid] = ok;
        if (b < p.batch && (b0 / kPlanThreads) % gridDim.x == blockIdx.x) {
            p.lens_out[b] = ok ? len + nw : len > 0 ? len : 0;
            if (!ok) plan_flag(p, SANTA_ERR_PAGES);
        }
        if (blockIdx.x == 0) {
            const unsigned a = __reduce_add_sync(kFull, ok ? unsigned(need) : 0u);
            const unsigned c = __reduce_add_sync(kFull, ok ? unsigned(n_tok) : 0u);
            if ((tid & 31) == 0) {
                atomicAdd(&s_sum[0], a);
                atomicAdd(&s_sum[1], c);
            }
        }
        __syncthreads();  // the arrays above are complete
        const int nb = min(kPlanThreads, p.batch - b0);
        for (long long i = me; i < tile_page; i += all) {
            const int s = upper(s_page, nb, i);
            if (!s_ok[s]) continue;
            const int k = int(i - (s > 0 ? s_page[s - 1] : 0));
            p.page_table[(size_t)(b0 + s) * p.max_pages + s_have[s] + k] = p.free_pages[page0 + i];
        }
        // tokens tok0 .. tok0 + tile_tok - 1, by groups of four that start at a multiple of four
        const long long row_end = min(tok0 + tile_tok, (long long)p.max_tokens);
        for (long long i0 = (tok0 & ~3LL) + 4 * me; i0 < row_end; i0 += 4 * all) {
            long long slot[4];
            int pos[4];
            int s = upper(s_tok, nb, i0 > tok0 ? i0 - tok0 : 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                slot[j] = -1;
                pos[j] = 0;
                const long long i = i0 + j - tok0;
                if (i0 + j >= row_end || i < 0) continue;
                while (s_tok[s] <= i) ++s;  // ends: i < tile_tok
                if (!s_ok[s]) continue;
                pos[j] = s_len[s] + int(i - (s > 0 ? s_tok[s - 1] : 0));
                const int pg = page_of(pos[j], p), fresh = pg - s_have[s];
                const int id = fresh >= 0 ? load(p.free_pages + page0 + (s > 0 ? s_page[s - 1] : 0) + fresh)
                                          : p.page_table[(size_t)(b0 + s) * p.max_pages + pg];
                if (id >= 0 && id < p.num_pages)
                    slot[j] = (long long)id * p.page_size + pos[j] - pg * p.page_size;
                else
                    plan_flag(p, SANTA_ERR_INDPTR);
            }
            if (i0 >= tok0 && i0 + 4 <= row_end) {
                reinterpret_cast<longlong2 *>(p.slot_map + i0)[0] = make_longlong2(slot[0], slot[1]);
                reinterpret_cast<longlong2 *>(p.slot_map + i0)[1] = make_longlong2(slot[2], slot[3]);
                *reinterpret_cast<int4 *>(p.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (i0 + j >= tok0 && i0 + j < row_end) {
                        p.slot_map[i0 + j] = slot[j];
                        p.positions[i0 + j] = pos[j];
                    }
            }
        }
        tok0 += tile_tok;
        page0 += tile_page;
        __syncthreads();
    }
    for (long long i = tok0 + me; i < p.max_tokens; i += all) {
        p.slot_map[i] = -1;
        p.positions[i] = 0;
    }
    if (me == 0) {
        p.counts[0] = int(s_sum[0]);  // the loop's last barrier is behind them
        p.counts[1] = int(s_sum[1]);
    }
}

}  // namespace

cudaError_t launch_page_plan(const PlanParams &plan, cudaStream_t stream) {
    PlanParams p = plan;
    int log = 0;
    while ((1LL << log) < p.page_size) ++log;
    if (log > 0) {  // 2^(31 + log) / d < 2^32
        p.magic = unsigned(((1ULL << (31 + log)) + p.page_size - 1) / p.page_size);
        p.shift = log - 1;
    }
    const int work = p.max_tokens > p.batch ? p.max_tokens : p.batch;
    int ctas = (work + kPlanThreads * 4 - 1) / (kPlanThreads * 4);
    ctas = ctas < 1 ? 1 : ctas > kPlanCtas ? kPlanCtas : ctas;
    return launch_kernel(page_plan_kernel, dim3(unsigned(ctas)), dim3(kPlanThreads), 0, stream, true, 0, false, p);
}

}  // namespace santa
