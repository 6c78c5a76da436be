// santa_norm_rope.cu -- per-head norms of q and k, the position rotation and the write
// of K and V into their cache rows, in one pass.
//
// For a head's vector x: y_i = x_i w_i / sqrt(mean(x^2) + eps) (skipped without a
// weight), then of the first rot_dim elements each pair (a, b) turns by the position's
// angle: (a c - b s, b c + a s).  A row (one head of one token) is held by D / 8 lanes, two
// chunks of 4 elements each, chosen so that a lane has both elements of its pairs: chunks l
// and l + rot/8 for the pairs (i, i + rot/2) (lanes behind rot/8 hold the rest of the row two
// chunks at a time), 8 neighbouring elements for the pairs (2i, 2i + 1).  A lane meets the
// same elements of every head, so it keeps their cosines, sines and weights in registers for
// all heads that it takes of the token: no shuffle but the norm's sum, no table read per head.
//
// Bound by memory: every row is read once and written once.  Lane rows take a token's rows in
// turn (queries, then keys, then values), kMany of them in flight; when there are not enough
// tokens to fill the GPU so, every lane row takes one row, and a warp passes by the kinds that
// it has no row of (one row per lane at 8191 tokens: 54 us; kMany at 777 tokens of 24 fp32 rows of
// 64: 8.3 us against 3.1).  8191 tokens, 32 query and 8 KV heads of 128 in bf16, 206 MB: 35.2 us =
// 5.8 TB/s, 0.86 of the copy rate.
//
// Several axes: a lane's four pairs may lie on four of them, so it takes its cosines and sines one by
// one from up to four rows of the table, once per token for all heads; 8191 tokens with norms and three
// axes in turn from pair to pair: 37.8 us.
#include "santa_rows.cuh"
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMany = 4;  // rows of a lane in flight

// Rows part, part + parts, ... below `end` of one token's `src` (row r at src + r D): norm
// (if there is a weight) and rotation (in lanes with `turns`) of q and k (kQK), and the store
// to dst (if `store`).  a0, a1: the lane's chunks.  Every part of a token makes the same number
// of iterations, so that the norm's shuffles are complete.
template <typename T, int D, bool kInter, bool kQK, int kAhead>
__device__ __forceinline__ void take_rows(const T *src, T *dst, const T *weight, float eps, int part, int parts, int end,
                                          bool turns, bool store, int a0, int a1, const float (&c)[4],
                                          const float (&s)[4]) {
    using E = Elems4<T>;
    using Raw = typename E::Raw;
    constexpr int kL = D / 8;
    if (kAhead == 1 && !__any_sync(kFull, store && part < end)) return;
    float w[8];
    if (kQK && weight) {
        float u[4], v[4];
        E::unpack(load(reinterpret_cast<const Raw *>(weight + a0)), u);
        E::unpack(load(reinterpret_cast<const Raw *>(weight + a1)), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = u[j], w[4 + j] = v[j];
    }
    for (int base = 0; base < end; base += parts * kAhead) {
        Raw ra[kAhead], rb[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = base + part + k * parts;
            const T *at = src + min(r, end - 1) * D;
            ra[k] = load(reinterpret_cast<const Raw *>(at + a0));
            rb[k] = load(reinterpret_cast<const Raw *>(at + a1));
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (base + k * parts >= end) break;
            const int r = base + part + k * parts;
            if constexpr (kQK) {
                float a[4], b[4];
                E::unpack(ra[k], a);
                E::unpack(rb[k], b);
                if (weight) {
                    float ss = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) ss = fmaf(a[j], a[j], fmaf(b[j], b[j], ss));
#pragma unroll
                    for (int o = 1; o < kL; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
                    const float inv = 1.f / sqrtf(ss / float(D) + eps);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a[j] *= inv * w[j];
                        b[j] *= inv * w[4 + j];
                    }
                }
                if (turns) {
                    if constexpr (kInter) {  // (a0, a1), (a2, a3), (b0, b1), (b2, b3)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float x = a[2 * j], y = a[2 * j + 1], u = b[2 * j], v = b[2 * j + 1];
                            a[2 * j] = fmaf(x, c[j], -y * s[j]);
                            a[2 * j + 1] = fmaf(y, c[j], x * s[j]);
                            b[2 * j] = fmaf(u, c[2 + j], -v * s[2 + j]);
                            b[2 * j + 1] = fmaf(v, c[2 + j], u * s[2 + j]);
                        }
                    } else {  // (a_j, b_j)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = a[j], y = b[j];
                            a[j] = fmaf(x, c[j], -y * s[j]);
                            b[j] = fmaf(y, c[j], x * s[j]);
                        }
                    }
                }
                ra[k] = E::pack(a);
                rb[k] = E::pack(b);
            }
            if (store && r < end) {
                T *to = dst + r * D;
                *reinterpret_cast<Raw *>(to + a0) = ra[k];
                *reinterpret_cast<Raw *>(to + a1) = rb[k];
            }
        }
    }
}

// A lane row takes the rows part, part + parts, ... of one token's Hq queries, Hkv keys and Hkv values.
// kAxes: a position per axis, and an axis per pair (two bits each, the lane's four in axis4[l]).
template <typename T, int D, bool kInter, int kAhead, bool kAxes>
__global__ void __launch_bounds__(kRopeThreads, sizeof(T) == 2 ? 4 : 3)
    norm_rope_kernel(const __grid_constant__ RopeParams p, int parts) {
    constexpr int kL = D / 8;
    const int l = threadIdx.x % kL;
    const long long row = ((long long)blockIdx.x * kRopeThreads + threadIdx.x) / kL;
    const long long t_ = row >> 31 ? row / parts : (long long)(unsigned(row) / unsigned(parts));
    const int part = int(row - t_ * parts);
    const bool live = t_ < p.tokens;  // whole lane rows; the others keep the warp's shuffles complete
    const long long t = live ? t_ : p.tokens - 1;
    // the lane's chunks, and the first pair's index
    const int eighth = p.rot_dim / 8;
    const bool turns = kInter ? 8 * l < p.rot_dim : l < eighth;
    const int a0 = kInter || !turns ? 8 * l : 4 * l, a1 = kInter || !turns ? 8 * l + 4 : 4 * l + 4 * eighth;
    pdl_wait();
    pdl_launch_dependents();

    auto checked = [&](int pos) {
        if (pos < 0 || pos >= p.max_pos) {
            if (p.err && live) atomicOr(p.err, SANTA_ERR_POSITION);
            pos = pos < 0 ? 0 : p.max_pos - 1;
        }
        return pos;
    };
    long long slot = p.slot_map ? load(p.slot_map + t) : t;
    if (slot >= p.total_tokens) {
        if (p.err && live) atomicOr(p.err, SANTA_ERR_SLOT);
        slot = -1;
    }
    float c[4] = {}, s[4] = {};
    if constexpr (kAxes) {
        int pos[4] = {};
#pragma unroll
        for (int a = 0; a < 4; ++a)
            if (a < p.axes) pos[a] = checked(load(p.positions + a * p.axis_stride + t));
        if (turns) {
            const float *cs = p.cos_sin + 4 * l;
            const unsigned ax = p.axis4[l];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned a = ax >> (2 * j) & 3;
                const float *at = cs + (size_t)(a < 2 ? a == 0 ? pos[0] : pos[1] : a == 2 ? pos[2] : pos[3]) * p.rot_dim + j;
                c[j] = load(at);
                s[j] = load(at + p.rot_dim / 2);
            }
        }
    } else {
        const int pos = checked(load(p.positions + t));
        if (turns) {
            const float *cs = p.cos_sin + (size_t)pos * p.rot_dim + 4 * l;
            const float4 u = load(reinterpret_cast<const float4 *>(cs));
            const float4 v = load(reinterpret_cast<const float4 *>(cs + p.rot_dim / 2));
            c[0] = u.x, c[1] = u.y, c[2] = u.z, c[3] = u.w;
            s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
        }
    }
    const int nq = p.q ? p.Hq : 0, nk = p.k ? p.Hkv : 0, nv = p.v ? p.Hkv : 0;
    // row r of the token goes to part r mod parts, counted through q, k and v
    if (nq > 0)
        take_rows<T, D, kInter, true, kAhead>(static_cast<const T *>(p.q) + t * p.q_stride, static_cast<T *>(p.q_out) + t * nq * D,
                                      static_cast<const T *>(p.q_weight), p.eps, part, parts, nq, turns, live, a0, a1, c, s);
    const bool cached = live && slot >= 0;
    const size_t at = (size_t)(slot < 0 ? 0 : slot) * p.Hkv * D;
    if (nk > 0) {
        const int k0 = (part + parts - nq % parts) % parts;
        take_rows<T, D, kInter, true, kAhead>(static_cast<const T *>(p.k) + t * p.k_stride, static_cast<T *>(p.k_cache) + at,
                                      static_cast<const T *>(p.k_weight), p.eps, k0, parts, nk, turns, cached, a0, a1, c, s);
    }
    if (nv > 0) {
        const int v0 = (part + parts - (nq + nk) % parts) % parts;
        take_rows<T, D, kInter, false, kAhead>(static_cast<const T *>(p.v) + t * p.v_stride, static_cast<T *>(p.v_cache) + at,
                                       static_cast<const T *>(nullptr), 0.f, v0, parts, nv, false, cached, a0, a1, c, s);
    }
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams &p, int dtype, int d, cudaStream_t stream) {
    const int rows = (p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (p.v ? p.Hkv : 0);
    // a third of the lanes that the SMs hold (2048 threads each): a lane row then pays for its
    // table row and weights over more rows.  With all of them, 48 rows of 128 per token: 1000
    // tokens 11.8 us instead of 7.0, 4000 21.8 instead of 18.9, 8191 36.1 instead of 35.4; with a
    // sixth: 4000 tokens 24.8.
    int parts = 1;
    while (parts < rows && (long long)p.tokens * parts * (d / 8) < 152LL * 640) parts *= 2;
    const bool one = parts * kMany > rows;
    if (one) parts = rows;
    const long long threads = (long long)p.tokens * parts * (d / 8);
    const long long ctas = (threads + kRopeThreads - 1) / kRopeThreads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        return launch_kernel(kern, dim3(unsigned(ctas)), dim3(kRopeThreads), 0, stream, true, 0, false, p, parts);
    };
    auto pick = [&](auto inter, auto ahead, auto axes) {
        constexpr bool kInter = decltype(inter)::value, kAx = decltype(axes)::value;
        constexpr int kA = decltype(ahead)::value;
        if (dtype == SANTA_BF16)
            return d == 128 ? go(norm_rope_kernel<uint16_t, 128, kInter, kA, kAx>)
                            : go(norm_rope_kernel<uint16_t, 64, kInter, kA, kAx>);
        return d == 128 ? go(norm_rope_kernel<float, 128, kInter, kA, kAx>) : go(norm_rope_kernel<float, 64, kInter, kA, kAx>);
    };
    auto pick_ahead = [&](auto inter, auto axes) {
        return one ? pick(inter, std::integral_constant<int, 1>(), axes) : pick(inter, std::integral_constant<int, kMany>(), axes);
    };
    if (p.axes)
        return p.interleaved ? pick_ahead(std::true_type(), std::true_type()) : pick_ahead(std::false_type(), std::true_type());
    return p.interleaved ? pick_ahead(std::true_type(), std::false_type()) : pick_ahead(std::false_type(), std::false_type());
}

}  // namespace santa
