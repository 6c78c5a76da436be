// santa_split.cuh -- how the visible keys of a batch are shared out over the GPU, and how
// the pieces of a head are joined again.
//
// The unit of work is a block of 32 keys of one (sequence, KV head).  A sequence shows
// its first ceil(s / 32) blocks and those from the one that holds the window's first key
// on (all of them where the two meet); its blocks are numbered through.  The units of the
// batch in the order (sequence, KV head, block) are cut into equal contiguous stretches,
// one per warp of the grid, so that every warp has the same number of units, to one,
// whatever the lengths are; lengths are read on the device, and each warp works out its
// own stretch.  A warp keeps an online softmax (M, Z, O) per query head and closes it
// when its stretch leaves a head:
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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A head of the walk: the visible blocks of (sequence b, KV head kvh), units u0 .. u0 + nb - 1.
struct Head {
    int b, kvh, nb;
    long long u0;
    long long start;  // the sequence's first row (contiguous cache)
    Visible vis;
    int nsb, wb0;     // sink blocks; the window's first block
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
    h.b = b;
    set_blocks(h, seq_bounds<kPaged>(sp.p, b, &h.start), sp);
}

// Stretch c of `parts` equal ones of X units starts at: (the first X mod parts are one longer)
__device__ __forceinline__ long long stretch_start(long long X, int parts, int c) {
    const long long q = X / parts, r = X - q * parts;
    return q * c + (c < r ? c : r);
}
// The stretch that unit x lies in.
__device__ __forceinline__ int stretch_of(long long X, int parts, long long x) {
    const long long q = X / parts, r = X - q * parts, big = r * (q + 1);
    return int(x < big ? x / (q + 1) : r + (x - big) / (q > 0 ? q : 1));
}

// What a CTA's warps share.
template <int NW>
struct SplitShared {
    float M[2 * NW][kMaxGroup], Z[2 * NW][kMaxGroup];  // pieces 2w (first head of warp w), 2w + 1 (last)
    long long u0[2 * NW];                              // the piece's head; -1: no piece
    int b[2 * NW], kvh[2 * NW], nb[2 * NW];
    long long inc_u0[2];                               // the CTA's heads that others share: first, last
    int inc_b[2], inc_kvh[2], inc_nb[2], inc_parts[2], last[2];
    long long x0[NW];                                  // plan of a large batch: where the warps start
    long long prefix[NW];
    int start_b[NW];
    long long scan[NW + 1];
};

// A warp's place in the walk.
struct Walk {
    long long x, x_end;     // next unit, end of the stretch
    long long cta0, cta1;   // the CTA's stretch
    long long X;
    int ctas;               // CTAs that have a stretch
    int n;                  // block of `head`
    Head head;
};

__device__ __forceinline__ void zero_row(const Params &p, int b) {
    float4 *o = reinterpret_cast<float4 *>(p.out + size_t(b) * p.Hq * p.D);
    for (int i = threadIdx.x; i < p.Hq * p.D / 4; i += blockDim.x) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// Finds the warp's stretch and its first unit; zeroes the rows of sequences without a key
// (each by one CTA).  False: the warp has no unit.  Every thread of the CTA calls it.
template <int NW, bool kPaged>
__device__ __forceinline__ bool plan_walk(const SplitParams &sp, SplitShared<NW> &sh, Walk &w) {
    const Params &p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long total = 0, prefix = 0;
    int b = -1;
    auto ranges = [&]() {
        w.X = total * p.Hkv;
        const long long most = (w.X + kMinUnitsPerCta - 1) / kMinUnitsPerCta;
        w.ctas = most < (long long)gridDim.x ? int(most) : int(gridDim.x);
        if ((int)blockIdx.x >= w.ctas) {
            w.x = w.x_end = w.cta0 = w.cta1 = w.X;
            return;
        }
        w.cta0 = stretch_start(w.X, w.ctas, blockIdx.x);
        w.cta1 = stretch_start(w.X, w.ctas, blockIdx.x + 1);
        const int len = int(w.cta1 - w.cta0);
        w.x = w.cta0 + stretch_start(len, NW, warp);
        w.x_end = w.cta0 + stretch_start(len, NW, warp + 1);
    };
    if (p.B <= 128) {  // every warp scans for itself: no barrier
        int nb[4];
        long long end[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            nb[k] = 0;
            if (32 * k < p.B) {
                Head h;
                if (32 * k + lane < p.B) {
                    load_head<kPaged>(h, sp, 32 * k + lane);
                    nb[k] = h.nb;
                }
                unsigned empty = __ballot_sync(kFull, 32 * k + lane < p.B && nb[k] == 0);
                while (empty) {
                    const int e = 32 * k + __ffs(empty) - 1;
                    empty &= empty - 1;
                    if (e % gridDim.x == blockIdx.x) zero_row(p, e);
                }
                long long v = nb[k];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long u = __shfl_up_sync(kFull, v, o);
                    if (lane >= o) v += u;
                }
                end[k] = total + v;
                total = __shfl_sync(kFull, end[k], 31);
            }
        }
        ranges();
        if (w.x < w.x_end) {
#pragma unroll
            for (int k = 3; k >= 0; --k)
                if (32 * k < p.B) {
                    const unsigned past = __ballot_sync(kFull, 32 * k + lane < p.B && end[k] * p.Hkv > w.x);
                    if (past) {
                        const int l = __ffs(past) - 1;
                        b = 32 * k + l;
                        prefix = __shfl_sync(kFull, end[k] - nb[k], l);
                    }
                }
        }
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
            Head h;
            h.nb = 0;
            if (b0 + (int)threadIdx.x < p.B) load_head<kPaged>(h, sp, b0 + threadIdx.x);
            long long all;
            block_scan(h.nb, &all);
            total += all;
        }
        ranges();
        if (lane == 0) {
            sh.x0[warp] = w.x < w.x_end ? w.x : -1;
            sh.start_b[warp] = -1;
        }
        long long carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += NT) {
            Head h;
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
    if (w.x >= w.x_end || b < 0) {
        w.x = w.x_end;
        return false;
    }
    load_head<kPaged>(w.head, sp, b);
    const long long rem = w.x - prefix * p.Hkv;
    w.head.kvh = int(rem / w.head.nb);
    w.n = int(rem - (long long)w.head.kvh * w.head.nb);
    w.head.u0 = w.x - w.n;
    return true;
}

// Moves to the next unit; false at the stretch's end.
template <bool kPaged>
__device__ __forceinline__ bool next_unit(const SplitParams &sp, Walk &w) {
    if (++w.x >= w.x_end) return false;
    if (++w.n < w.head.nb) return true;
    w.n = 0;
    w.head.u0 = w.x;
    if (++w.head.kvh < sp.p.Hkv) return true;
    w.head.kvh = 0;
    int b = w.head.b;
    do {
        load_head<kPaged>(w.head, sp, ++b);
    } while (w.head.nb == 0 && b + 1 < sp.p.B);
    return true;
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
// is the address of a piece's sums [G][D] in shared memory (sh.M, sh.Z beside them);
// `coef` room for ctas * G floats there, not overlapping the pieces' use after the barrier
// that follows them.  Every thread of the CTA calls it, after its warp's pieces are written.
template <int NW, int D, typename PieceAddr>
__device__ __forceinline__ void join_pieces(const SplitParams &sp, SplitShared<NW> &sh, const Walk &w, PieceAddr piece,
                                            float *coef, float *red) {
    const Params &p = sp.p;
    constexpr int kE = D / 32, NT = NW * 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = p.G;
    if (threadIdx.x < 2) sh.inc_u0[threadIdx.x] = -1;
    __syncthreads();
    // one (group of pieces of a head, query head) per warp at a time; a group begins at its first piece
    for (int item = warp; item < 2 * NW * G; item += NW) {
        const int i = item / G, h = item - i * G;
        const long long u0 = sh.u0[i];
        if (u0 < 0) continue;
        const bool in = lane < 2 * NW && sh.u0[lane < 2 * NW ? lane : 0] == u0;
        const unsigned members = __ballot_sync(kFull, in);
        if (__ffs(members) - 1 != i) continue;
        float m = in ? sh.M[lane][h] : -INFINITY;
        const float M = warp_max(m), Mref = M == -INFINITY ? 0.f : M;
        const float c = in ? ex2(m - Mref) : 0.f;
        const float Z = warp_sum(in ? sh.Z[lane][h] * c : 0.f);
        float o[kE];
#pragma unroll
        for (int e = 0; e < kE; ++e) o[e] = 0.f;
        for (unsigned left = members; left; left &= left - 1) {
            const int s = __ffs(left) - 1;
            const float cs = __shfl_sync(kFull, c, s);
            const float *src = piece(s) + h * D + lane * kE;
#pragma unroll
            for (int e = 0; e < kE; ++e) o[e] = fmaf(cs, src[e], o[e]);
        }
        if (u0 >= w.cta0 && u0 + sh.nb[i] <= w.cta1) {  // nobody else has a part
            const float inv = Z == 0.f ? 0.f : 1.f / Z;
            float *dst = p.out + (size_t(sh.b[i]) * p.Hq + sh.kvh[i] * G + h) * D + lane * kE;
#pragma unroll
            for (int e = 0; e < kE; ++e) dst[e] = Z == 0.f ? 0.f : o[e] * inv;
        } else {
            const int part = u0 <= w.cta0 ? 0 : 1;
            const size_t at = (size_t(blockIdx.x) * 2 + part) * G + h;
            float *dst = sp.part + at * D + lane * kE;
#pragma unroll
            for (int e = 0; e < kE; ++e) __stcg(dst + e, o[e]);
            if (lane == 0) {
                __stcg(sp.part_mz + at, make_float2(M, Z));
                if (h == 0) {
                    sh.inc_u0[part] = u0;
                    sh.inc_b[part] = sh.b[i];
                    sh.inc_kvh[part] = sh.kvh[i];
                    sh.inc_nb[part] = sh.nb[i];
                }
            }
            __threadfence();
        }
    }
    __syncthreads();
    if (threadIdx.x < 2) {
        const int k = threadIdx.x;
        sh.last[k] = 0;
        if (sh.inc_u0[k] >= 0) {
            const int first = stretch_of(w.X, w.ctas, sh.inc_u0[k]);
            const int parts = stretch_of(w.X, w.ctas, sh.inc_u0[k] + sh.inc_nb[k] - 1) - first + 1;
            sh.inc_parts[k] = parts;
            __threadfence();
            unsigned *cnt = sp.cnt + size_t(sh.inc_b[k]) * p.Hkv + sh.inc_kvh[k];
            if (atomicAdd(cnt, 1u) == unsigned(parts - 1)) {
                sh.last[k] = 1;
                *cnt = 0u;
            }
            __threadfence();
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        if (!sh.last[k]) continue;
        const int parts = sh.inc_parts[k], first = stretch_of(w.X, w.ctas, sh.inc_u0[k]);
        // part c of the head: the head is the first CTA's first one only if it starts its stretch
        const int slot0 = sh.inc_u0[k] <= stretch_start(w.X, w.ctas, first) ? 0 : 1;
        auto index = [&](int c) { return (size_t(first + c) * 2 + (c == 0 ? slot0 : 0)) * G; };
        for (int h = warp; h < G; h += NW) {
            float M = -INFINITY, Z = 0.f;
            for (int c = lane; c < parts; c += 32) M = fmaxf(M, __ldcg(sp.part_mz + index(c) + h).x);
            M = warp_max(M);
            const float Mref = M == -INFINITY ? 0.f : M;
            for (int c = lane; c < parts; c += 32) {
                const float2 mz = __ldcg(sp.part_mz + index(c) + h);
                const float f = ex2(mz.x - Mref);
                coef[c * G + h] = f;
                Z = fmaf(mz.y, f, Z);
            }
            Z = warp_sum(Z);
            __syncwarp();
            for (int c = lane; c < parts; c += 32) coef[c * G + h] = Z == 0.f ? 0.f : coef[c * G + h] / Z;
        }
        __syncthreads();
        // the sums: groups of G D / 4 threads take the parts in turn, then the groups in order
        const int cols = G * D / 4, groups = NT >= cols ? NT / cols : 1;
        for (int c0 = 0; c0 < cols; c0 += NT) {
            const int col = NT >= cols ? threadIdx.x % cols : c0 + threadIdx.x, grp = NT >= cols ? threadIdx.x / cols : 0;
            const bool on = grp < groups && col < cols;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (on) {
                const int h = col * 4 / D;
#pragma unroll 8
                for (int c = grp; c < parts; c += groups) {
                    const float f = coef[c * G + h];
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(sp.part + index(c) * D) + col);
                    acc.x = fmaf(f, v.x, acc.x);
                    acc.y = fmaf(f, v.y, acc.y);
                    acc.z = fmaf(f, v.z, acc.z);
                    acc.w = fmaf(f, v.w, acc.w);
                }
            }
            float4 *r4 = reinterpret_cast<float4 *>(red);
            if (groups > 1) {
                if (on) r4[grp * cols + col] = acc;
                __syncthreads();
                if (on && grp == 0)
                    for (int g = 1; g < groups; ++g) {
                        const float4 v = r4[g * cols + col];
                        acc.x += v.x;
                        acc.y += v.y;
                        acc.z += v.z;
                        acc.w += v.w;
                    }
            }
            if (on && grp == 0)
                reinterpret_cast<float4 *>(p.out + (size_t(sh.inc_b[k]) * p.Hq + sh.inc_kvh[k] * G) * D)[col] = acc;
        }
        __syncthreads();
    }
}

}  // namespace santa
