// santa_split.cuh -- how the visible keys of a batch are shared out over the GPU, and how
// the pieces of a head are joined again.
//
// The unit of work is a block of 32 keys of one (sequence, KV head).  A sequence shows
// its first ceil(s / 32) blocks and those from the one that holds the window's first key
// on (all of them where the two meet); its blocks are numbered through.  The units of the
// batch in the order (sequence, KV head, block) are cut into equal contiguous stretches,
// one per warp of the grid, so that every warp has the same number of units, to one,
// whatever the lengths are; lengths are read on the device, and each warp works out its
// own stretch.  (Where that costs more than it gives, kJoinUnits, each CTA takes one head
// instead, and nothing is joined across CTAs.)  A warp keeps an online softmax (M, Z, O) per
// query head and closes it when its stretch leaves a head:
//   - a head that lies within the stretch is finished by the warp itself;
//   - a head shared by warps of one CTA only is joined through shared memory;
//   - a head shared by CTAs: each CTA joins its warps' pieces, stores one part in the
//     workspace and counts itself in on the head's counter; the CTA that completes the
//     count joins the parts, and sets the counter back to zero.  No CTA ever waits for
//     another.
// Every join runs over the pieces in the order of the units, so results do not depend on
// timing.  M and the exponents are in base 2: x' = x log2(e).
#pragma once

#include "santa_tile.cuh"
#include "santa_visible.cuh"

namespace santa {

constexpr int kBlock = 32;         // keys per unit
constexpr int kMinUnitsPerCta = 4; // fewer CTAs than the grid has while a CTA would get less
// Joining a head's parts across CTAs costs about as much as a CTA's reading of this many
// units (4 us; a unit adds 0.14 to 0.16 us to a CTA's time, bf16 or 4-bit, d = 128; other
// dimensions and fp32 were not measured for this choice).  So when
// the heads are no more than the CTAs, each takes one head whole unless the longest head is
// longer than this and an equal share of all units together.  Batch 1, 8 KV heads, bf16, whole
// against split: 256 keys 6.2 / 8.9 us, 768 8.9 / 9.4, 1024 10.2 / 9.6, 2048 15.0 / 9.9; batch
// 16: 1024 keys 12.0 / 16.5, 2048 26.2 / 30.6.
constexpr int kJoinUnits = 28;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// An 8 x 8 matrix of 16-bit elements, two per lane, transposed over the warp.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A head of the walk: the visible blocks of (sequence b, KV head kvh), units u0 .. u0 + nb - 1.
struct Head {
    int b, kvh, nb;
    long long u0;
    int start;        // the sequence's first row (contiguous cache; rows fit 31 bits)
    Visible vis;
    int nsb, wb0;     // sink blocks; the window's first block
    bool began;       // the head begins in the warp's stretch
    __device__ __forceinline__ int first_key(int n) const { return kBlock * (n < nsb ? n : wb0 + n - nsb); }
};
__device__ __forceinline__ void set_blocks(Head &h, int L, const SplitParams &sp) {
    h.vis = visible(L, sp.window, sp.sinks);
    h.nsb = (h.vis.s + kBlock - 1) / kBlock;
    h.wb0 = h.vis.lo / kBlock;
    if (h.wb0 < h.nsb || h.vis.lo >= L) {  // the two meet, or all keys are sinks
        if (h.vis.lo < L) {
            h.nsb = 0;
            h.wb0 = 0;
        } else {
            h.wb0 = (L + kBlock - 1) / kBlock;
        }
    }
    h.nb = h.nsb + (L + kBlock - 1) / kBlock - h.wb0;
}
template <bool kPaged>
__device__ __forceinline__ void load_head(Head &h, const SplitParams &sp, int b) {
    long long start;
    h.b = b;
    set_blocks(h, seq_bounds<kPaged>(sp.p, b, &start), sp);
    h.start = int(start);
}

// a / b for a >= 0, b > 0: by 32 bits where they fit (the 64-bit division is a subroutine).
__device__ __forceinline__ long long divide(long long a, int b) {
    return a >> 31 ? a / b : (long long)(unsigned(a) / unsigned(b));
}
// Stretch c of `parts` equal ones of X units starts at: (the first X mod parts are one longer)
__device__ __forceinline__ long long stretch_start(long long X, int parts, int c) {
    const long long q = divide(X, parts), r = X - q * parts;
    return q * c + (c < r ? c : r);
}
// The stretch that unit x lies in.
__device__ __forceinline__ int stretch_of(long long X, int parts, long long x) {
    const long long q = divide(X, parts), r = X - q * parts, big = r * (q + 1);
    if (q >> 30) return int(x < big ? x / (q + 1) : r + (x - big) / q);
    return x < big ? int(divide(x, int(q) + 1)) : int(r + divide(x - big, q > 0 ? int(q) : 1));
}

// What a CTA's warps share.
template <int NW>
struct SplitShared {
    float M[2 * NW][kMaxGroup], Z[2 * NW][kMaxGroup];  // pieces 2w (first head of warp w), 2w + 1 (last)
    long long u0[2 * NW];                              // the piece's head; -1: no piece
    int b[2 * NW], kvh[2 * NW], nb[2 * NW];
    Head heads[NW][2];                                 // see Walk
    float coef[2 * NW][kMaxGroup];                     // weight of a piece in its head's sum
    int list[2 * NW + 1];                              // the pieces there are, in order
    int begin[2 * NW + 1];                             // where in `list` each head's pieces begin
    long long inc_u0[2];                               // the CTA's heads that others share: first, last
    int inc_b[2], inc_kvh[2], inc_first[2], inc_parts[2], last[2];
    long long X, cta0, cta1;                           // units of the batch; the CTA's stretch
    int ctas;                                          // CTAs that have a stretch
    long long x0[NW];                                  // plan of a large batch: where the warps start
    long long prefix[NW];
    int start_b[NW];
    long long scan[NW + 1];
};

// A warp's place in the walk.  Its head, and the one before it (which the block being
// computed may still belong to), lie in shared memory: they are looked at once per run of
// blocks, and would hold a dozen registers per thread.
struct Walk {
    int left;     // units of the stretch, this one included
    int n, run;   // block of the head; where its run of consecutive keys ends
    int key0;     // the block's first key
    int in_page;  // paged: where in its page the block begins
    int ahead;    // paged: the page table's next entry (loaded a page ahead of its use)
    int row;      // its first cache row; -1: a bad page id (flagged), its keys are dropped
    int sel;      // the head: heads[sel]
    Head *heads;  // [2], the warp's own
};

// Makes h the head of `slot`; every lane holds the same h.
__device__ __forceinline__ void put_head(Walk &w, int slot, const Head &h) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) w.heads[slot] = h;
    __syncwarp();
}
// The first cache row of a page, -1 (flagged) for a bad id.
__device__ __forceinline__ int page_row(const Params &p, int id) {
    if (id >= 0 && id < p.num_pages) return id * p.page_size;
    raise_flag(p, SANTA_ERR_INDPTR);
    return -1;
}
// Loads the table's entry behind the page of w.key0, if the row has one.
__device__ __forceinline__ void look_ahead(const Params &p, Walk &w, int b) {
    const int i = (w.key0 - w.in_page) / p.page_size + 1;
    w.ahead = i < p.max_pages ? load(p.page_table + (size_t)b * p.max_pages + i) : -1;
}
// The run and the row of block w.n of h, by the page table.
template <bool kPaged>
__device__ __forceinline__ void place(const SplitParams &sp, Walk &w, const Head &h) {
    const Params &p = sp.p;
    w.run = w.n < h.nsb ? h.nsb : h.nb;
    w.key0 = h.first_key(w.n);
    if constexpr (kPaged) {
        const int page = w.key0 / p.page_size;
        w.in_page = w.key0 - page * p.page_size;
        w.row = page_row(p, load(p.page_table + (size_t)h.b * p.max_pages + page));
        if (w.row >= 0) w.row += w.in_page;
        look_ahead(p, w, h.b);
    } else {
        w.row = h.start + w.key0;
    }
}
// Which of the 32 keys of the walk's block the query sees, a bit each.
__device__ __forceinline__ unsigned seen_bits(const Walk &w) {
    const Visible v = w.heads[w.sel].vis;
    const int key = w.key0 + (threadIdx.x & 31);
    return __ballot_sync(kFull, w.row >= 0 && key < v.L && (key < v.s || key >= v.lo));
}

__device__ __forceinline__ void zero_row(const Params &p, int b) {
    float4 *o = reinterpret_cast<float4 *>(p.out + size_t(b) * p.Hq * p.D);
    for (int i = threadIdx.x; i < p.Hq * p.D / 4; i += blockDim.x) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Finds the warp's stretch and its first unit; zeroes the rows of sequences without a key
// (each by one CTA).  1: the walk stands on the warp's first unit; 0: the warp has none; -1: the
// CTA has none.  Every thread of the CTA calls it.
template <int NW, bool kPaged>
__device__ __forceinline__ int plan_walk(const SplitParams &sp, SplitShared<NW> &sh, Walk &w) {
    const Params &p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long total = 0, prefix = 0, x = 0;
    int b = -1;
    w.left = 0;
    int ctas;  // that have a stretch
    // The CTA's stretch is cta0 .. cta1 - 1; the warp's, an equal part of it.
    auto take = [&](long long X, long long cta0, long long cta1) {
        const long long from = stretch_start(cta1 - cta0, NW, warp);
        x = cta0 + from;
        w.left = int(stretch_start(cta1 - cta0, NW, warp + 1) - from);
        if (threadIdx.x == 0) {
            sh.X = X;
            sh.cta0 = cta0;
            sh.cta1 = cta1;
            sh.ctas = ctas;
        }
    };
    auto equal_stretches = [&]() {
        const long long X = total * p.Hkv, most = (X + kMinUnitsPerCta - 1) / kMinUnitsPerCta;
        ctas = most < (long long)gridDim.x ? int(most) : int(gridDim.x);
        if ((int)blockIdx.x < ctas) take(X, stretch_start(X, ctas, blockIdx.x), stretch_start(X, ctas, blockIdx.x + 1));
    };
    Head h;
    if (sp.narrow) {  // at most 128 sequences, units counted in 31 bits: every warp scans for itself, no barrier
        int nb[4], len[4], from[4], end[4], most = 0, sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            nb[k] = len[k] = from[k] = 0;
            if (32 * k < p.B) {
                if (32 * k + lane < p.B) {
                    load_head<kPaged>(h, sp, 32 * k + lane);
                    nb[k] = h.nb;
                    len[k] = h.vis.L;
                    from[k] = h.start;
                }
                most = max(most, nb[k]);
                unsigned empty = __ballot_sync(kFull, 32 * k + lane < p.B && nb[k] == 0);
                while (empty) {
                    const int e = 32 * k + __ffs(empty) - 1;
                    empty &= empty - 1;
                    if (e % gridDim.x == blockIdx.x) zero_row(p, e);
                }
                int v = nb[k];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    if (o >= p.B) break;
                    const int u = __shfl_up_sync(kFull, v, o);
                    if (lane >= o) v += u;
                }
                end[k] = sum + v;
                sum = __shfl_sync(kFull, end[k], min(31, p.B - 32 * k - 1));
            }
        }
        const unsigned X = unsigned(sum) * p.Hkv, heads = unsigned(p.B) * p.Hkv;
        unsigned cta0 = 0, size = 0;  // the CTA's stretch
        if (heads <= gridDim.x && __reduce_max_sync(kFull, unsigned(most)) <= kJoinUnits + X / gridDim.x) {  // a CTA per head
            ctas = int(heads);
            if (blockIdx.x >= heads) return -1;
            b = blockIdx.x / p.Hkv;
            int e = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (b / 32 == k) {
                    size = unsigned(__shfl_sync(kFull, nb[k], b % 32));
                    e = __shfl_sync(kFull, end[k], b % 32);
                }
            if (size == 0) return -1;
            cta0 = (unsigned(e) - size) * p.Hkv + (blockIdx.x - unsigned(b) * p.Hkv) * size;
        } else {
            const unsigned parts = min(gridDim.x, (X + kMinUnitsPerCta - 1) / kMinUnitsPerCta);
            ctas = int(parts);
            if (blockIdx.x >= parts) return -1;
            const unsigned q = X / parts, r = X - q * parts;  // as stretch_start
            cta0 = q * blockIdx.x + min(blockIdx.x, r);
            size = q + (blockIdx.x < r ? 1 : 0);
        }
        const unsigned q = size / NW, r = size - q * NW;
        const unsigned at = cta0 + q * warp + min(unsigned(warp), r);
        x = at;
        w.left = int(q + (unsigned(warp) < r ? 1 : 0));
        if (threadIdx.x == 0) {
            sh.X = X;
            sh.cta0 = cta0;
            sh.cta1 = (long long)cta0 + size;
            sh.ctas = ctas;
        }
        if (w.left <= 0) return 0;
#pragma unroll
        for (int k = 3; k >= 0; --k)
            if (32 * k < p.B) {
                const unsigned past = __ballot_sync(kFull, 32 * k + lane < p.B && unsigned(end[k]) * p.Hkv > at);
                if (past) {
                    const int l = __ffs(past) - 1;
                    b = 32 * k + l;
                    prefix = __shfl_sync(kFull, end[k] - nb[k], l);
                    h.start = __shfl_sync(kFull, from[k], l);
                    h.vis.L = __shfl_sync(kFull, len[k], l);
                }
            }
        h.b = b;
        set_blocks(h, h.vis.L, sp);
    } else {
        constexpr int NT = NW * 32;
        auto block_scan = [&](long long v, long long *all) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += u;
            }
            __syncthreads();
            if (lane == 31) sh.scan[warp] = v;
            __syncthreads();
            long long before = 0, sum = 0;
            for (int i = 0; i < NW; ++i) {
                const long long s = sh.scan[i];
                if (i < warp) before += s;
                sum += s;
            }
            *all = sum;
            return v + before;
        };
        for (int b0 = 0; b0 < p.B; b0 += NT) {
            h.nb = 0;
            if (b0 + (int)threadIdx.x < p.B) load_head<kPaged>(h, sp, b0 + threadIdx.x);
            long long all;
            block_scan(h.nb, &all);
            total += all;
        }
        equal_stretches();
        if (lane == 0) {
            sh.x0[warp] = w.left > 0 ? x : -1;
            sh.start_b[warp] = -1;
        }
        long long carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += NT) {
            h.nb = 0;
            const int mine = b0 + threadIdx.x;
            if (mine < p.B) load_head<kPaged>(h, sp, mine);
            long long all;
            const long long end = carry + block_scan(h.nb, &all);  // its barriers publish x0 and start_b too
            if (mine < p.B)
                for (int i = 0; i < NW; ++i)
                    if (sh.x0[i] >= (end - h.nb) * p.Hkv && sh.x0[i] < end * p.Hkv) {
                        sh.start_b[i] = mine;
                        sh.prefix[i] = end - h.nb;
                    }
            carry += all;
            // the rows of empty sequences, found a second time by the whole CTA
            for (int e = b0 + int((blockIdx.x + gridDim.x - b0 % gridDim.x) % gridDim.x); e < min(p.B, b0 + NT);
                 e += gridDim.x) {
                Head g;
                load_head<kPaged>(g, sp, e);
                if (g.nb == 0) zero_row(p, e);
            }
        }
        __syncthreads();
        b = sh.start_b[warp];
        prefix = sh.prefix[warp];
    }
    if ((int)blockIdx.x >= ctas) return -1;
    if (w.left <= 0 || b < 0) {
        w.left = 0;
        return 0;
    }
    if (!sp.narrow) load_head<kPaged>(h, sp, b);
    const long long rem = x - prefix * p.Hkv;
    h.kvh = int(divide(rem, h.nb));
    w.n = int(rem - (long long)h.kvh * h.nb);
    h.u0 = x - w.n;
    h.began = w.n == 0;
    w.sel = 0;
    w.heads = sh.heads[warp];
    place<kPaged>(sp, w, h);
    put_head(w, 0, h);
    return 1;
}

// Moves to the next unit.  0: the stretch has ended; 1: the next block of the head; 2: of
// another head (w.sel has changed).
template <bool kPaged>
__device__ __forceinline__ int next_unit(const SplitParams &sp, Walk &w) {
    if (--w.left <= 0) return 0;
    if (++w.n < w.run) {
        w.key0 += kBlock;
        if constexpr (!kPaged) {
            w.row += kBlock;
            return 1;
        } else {
            w.in_page += kBlock;
            if (w.in_page < sp.p.page_size) {
                if (w.row >= 0) w.row += kBlock;
            } else {
                w.in_page = 0;
                w.row = page_row(sp.p, w.ahead);
                look_ahead(sp.p, w, w.heads[w.sel].b);
            }
            return 1;
        }
    }
    Head h = w.heads[w.sel];
    if (w.n < h.nb) {  // from the sinks to the window
        place<kPaged>(sp, w, h);
        return 1;
    }
    w.n = 0;
    h.u0 += h.nb;
    h.began = true;
    if (++h.kvh >= sp.p.Hkv) {
        h.kvh = 0;
        int b = h.b;
        do {
            load_head<kPaged>(h, sp, ++b);
        } while (h.nb == 0 && b + 1 < sp.p.B);
    }
    place<kPaged>(sp, w, h);
    w.sel ^= 1;
    put_head(w, w.sel, h);
    return 2;
}

// Notes that piece `slot` belongs to `h`.  One lane.
template <int NW>
__device__ __forceinline__ void note_piece(SplitShared<NW> &sh, int slot, const Head &h) {
    sh.u0[slot] = h.u0;
    sh.b[slot] = h.b;
    sh.kvh[slot] = h.kvh;
    sh.nb[slot] = h.nb;
}

// Joins the CTA's pieces, and the parts of the heads that this CTA completes.  `piece(slot)`
// is the address of a piece's sums [G][D] in shared memory (sh.M, sh.Z beside them); `room`
// is shared memory for kSplitCtaBound * G floats and a float4 per thread, which may overlap
// the pieces.  Every thread of the CTA calls it, after its warp's pieces are written.
template <int NW, int D, typename PieceAddr>
__device__ __forceinline__ void join_pieces(const SplitParams &sp, SplitShared<NW> &sh, PieceAddr piece,
                                            float *room) {
    static_assert(2 * NW <= 32, "a lane per piece");
    const Params &p = sp.p;
    constexpr int NT = NW * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.G;
    if (threadIdx.x < 2) sh.inc_u0[threadIdx.x] = -1;
    __syncthreads();
    const long long cta0 = sh.cta0, cta1 = sh.cta1;
    // the pieces there are, and where each head's begin (every warp finds the same)
    const long long my_u0 = lane < 2 * NW ? sh.u0[lane] : -1;
    const unsigned valid = __ballot_sync(kFull, my_u0 >= 0);
    // pieces come in the order of the units, so a head's are neighbours among those there are
    const unsigned below = valid & ((1u << lane) - 1);
    const long long before = __shfl_sync(kFull, my_u0, below ? 31 - __clz(below) : lane);
    const unsigned heads = __ballot_sync(kFull, my_u0 >= 0 && (!below || before != my_u0));
    const int n_heads = __popc(heads);
    if (warp == 0) {
        const int at = __popc(below);
        if (my_u0 >= 0) sh.list[at] = lane;
        if (heads >> lane & 1) sh.begin[__popc(heads & ((1u << lane) - 1))] = at;
        if (lane == 0) sh.begin[n_heads] = __popc(valid);
    }
    for (int item = warp; item < n_heads * G; item += NW) {
        const int k = item / G, h = item - k * G;
        unsigned rest = heads;
        for (int q = 0; q < k; ++q) rest &= rest - 1;
        const int i = __ffs(rest) - 1;  // the head's first piece
        const long long u0 = __shfl_sync(kFull, my_u0, i);
        const bool in = my_u0 == u0;
        const float m = in ? sh.M[lane][h] : -INFINITY;
        const float M = warp_max(m), Mref = M == -INFINITY ? 0.f : M;
        float c = in ? ex2(m - Mref) : 0.f;
        const float Z = warp_sum(in ? sh.Z[lane][h] * c : 0.f);
        if (u0 >= cta0 && u0 + sh.nb[i] <= cta1) {  // nobody else has a part
            c = Z == 0.f ? 0.f : c / Z;
        } else if (lane == 0) {
            const int part = u0 <= cta0 ? 0 : 1;
            __stcg(sp.part_mz + (size_t(blockIdx.x) * 2 + part) * G + h, make_float2(M, Z));
            if (h == 0) {
                sh.inc_u0[part] = u0;
                sh.inc_b[part] = sh.b[i];
                sh.inc_kvh[part] = sh.kvh[i];
                const int first = stretch_of(sh.X, sh.ctas, u0);
                sh.inc_first[part] = first;
                sh.inc_parts[part] = stretch_of(sh.X, sh.ctas, u0 + sh.nb[i] - 1) - first + 1;
            }
        }
        if (in) sh.coef[lane][h] = c;
    }
    __syncthreads();
    const int cols = G * D / 4;  // float4 columns of a head's sums
    for (int task = threadIdx.x; task < n_heads * cols; task += NT) {
        const int k = task / cols, col = task - k * cols, h = col / (D / 4);
        const int j0 = sh.begin[k], j1 = sh.begin[k + 1], i = sh.list[j0];
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int j = j0; j < j1; ++j) {
            const int s = sh.list[j];
            const float c = sh.coef[s][h];
            const float4 v = reinterpret_cast<const float4 *>(piece(s))[col];
            o.x = fmaf(c, v.x, o.x);
            o.y = fmaf(c, v.y, o.y);
            o.z = fmaf(c, v.z, o.z);
            o.w = fmaf(c, v.w, o.w);
        }
        const long long u0 = sh.u0[i];
        if (u0 >= cta0 && u0 + sh.nb[i] <= cta1) {
            reinterpret_cast<float4 *>(p.out + (size_t(sh.b[i]) * p.Hq + sh.kvh[i] * G) * D)[col] = o;
        } else {
            const int part = u0 <= cta0 ? 0 : 1;
            __stcg(reinterpret_cast<float4 *>(sp.part + (size_t(blockIdx.x) * 2 + part) * G * D) + col, o);
        }
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        const int k = threadIdx.x;
        sh.last[k] = 0;
        if (sh.inc_u0[k] >= 0) {
            // the CTA's part is visible (the barrier above, this fence) before it is counted
            __threadfence();
            unsigned *cnt = sp.cnt + size_t(sh.inc_b[k]) * p.Hkv + sh.inc_kvh[k];
            const unsigned end = unsigned(sh.inc_parts[k] - 1);
            if (atomicInc(cnt, end) == end) {  // which sets it back to 0
                sh.last[k] = 1;
                __threadfence();  // the others' parts are read after their counts
            }
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (!sh.last[k]) continue;
        const int parts = sh.inc_parts[k], first = sh.inc_first[k];
        // the head is its first CTA's first one only if it starts that CTA's stretch
        const int slot0 = sh.inc_u0[k] <= stretch_start(sh.X, sh.ctas, first) ? 0 : 1;
        auto index = [&](int c) { return (size_t(first + c) * 2 + (c == 0 ? slot0 : 0)) * G; };
        // groups of threads take the parts in turn, a float4 column per thread (cols of them in
        // passes of at most NT); their first rows are requested before the coefficients are known
        for (int col0 = 0; col0 < cols; col0 += NT) {
            const int width = min(cols - col0, NT), groups = NT / width;
            const int grp = threadIdx.x / width, col = col0 + threadIdx.x - grp * width;
            const bool on = grp < groups;
            constexpr int kAhead = 8;
            float4 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int c = grp + u * groups;
                v[u] = on && c < parts ? __ldcg(reinterpret_cast<const float4 *>(sp.part + index(c) * D) + col)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float *coef = room;
            for (int h = warp; h < G && col0 == 0; h += NW) {
                constexpr int kPer = (kSplitCtaBound + 31) / 32;
                float2 mz[kPer];
                float M = -INFINITY, Z = 0.f;
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int c = lane + 32 * u;
                    mz[u] = c < parts ? __ldcg(sp.part_mz + index(c) + h) : make_float2(-INFINITY, 0.f);
                    M = fmaxf(M, mz[u].x);
                }
                M = warp_max(M);
                const float Mref = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    mz[u].x = ex2(mz[u].x - Mref);
                    Z = fmaf(mz[u].y, mz[u].x, Z);
                }
                Z = warp_sum(Z);
                const float inv = Z == 0.f ? 0.f : 1.f / Z;
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const int c = lane + 32 * u;
                    if (c < parts) coef[c * G + h] = Z == 0.f ? 0.f : mz[u].x * inv;
                }
            }
            __syncthreads();
            const int h = col / (D / 4);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int c = grp + u * groups;
                    const float f = c < parts ? coef[c * G + h] : 0.f;
                    acc.x = fmaf(f, v[u].x, acc.x);
                    acc.y = fmaf(f, v[u].y, acc.y);
                    acc.z = fmaf(f, v[u].z, acc.z);
                    acc.w = fmaf(f, v[u].w, acc.w);
                }
#pragma unroll 8
                for (int c = grp + kAhead * groups; c < parts; c += groups) {
                    const float f = coef[c * G + h];
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(sp.part + index(c) * D) + col);
                    acc.x = fmaf(f, x.x, acc.x);
                    acc.y = fmaf(f, x.y, acc.y);
                    acc.z = fmaf(f, x.z, acc.z);
                    acc.w = fmaf(f, x.w, acc.w);
                }
            }
            float4 *red = reinterpret_cast<float4 *>(room + kSplitCtaBound * kMaxGroup);
            if (groups > 1) {
                if (on && grp > 0) red[(grp - 1) * width + col - col0] = acc;
                __syncthreads();
                if (grp == 0)
                    for (int g = 1; g < groups; ++g) {
                        const float4 x = red[(g - 1) * width + col - col0];
                        acc.x += x.x;
                        acc.y += x.y;
                        acc.z += x.z;
                        acc.w += x.w;
                    }
            }
            if (grp == 0)
                reinterpret_cast<float4 *>(p.out + (size_t(sh.inc_b[k]) * p.Hq + sh.inc_kvh[k] * G) * D)[col] = acc;
            __syncthreads();
        }
    }
}

}  // namespace santa
