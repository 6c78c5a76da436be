// santa_norm_rope.cu -- per-head norms of q and k, the position rotation and the write
// of K and V into their cache rows, in one pass.
//
// For a head's vector x: y_i = x_i w_i / sqrt(mean(x^2) + eps) (skipped without a
// weight), then of the first rot_dim elements each pair (a, b) turns by the position's
// angle: (a c - b s, b c + a s).  A row (one head of one token) is held by D / 8 lanes,
// 8 consecutive elements each, so a lane meets the same 8 elements of every head: it
// keeps their weights, cosines and sines in registers for all heads that it takes of the
// token.  Pairs (i, i + rot/2) lie in lanes rot/16 apart (one shuffle per element; rot
// is a multiple of 16), pairs (2i, 2i + 1) in one lane.
//
// Bound by memory: every row is read once and written once.
#include "santa_rows.cuh"
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kRopeThreads = 256;

// One thread row of D / 8 lanes takes the rows part, part + parts, ... of one token:
// its Hq queries, then its Hkv keys, then its Hkv values.
template <typename T, int D>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams p, int parts) {
    constexpr int kL = D / 8;  // lanes of a row
    const int l = threadIdx.x % kL;
    const long long row = ((long long)blockIdx.x * kRopeThreads + threadIdx.x) / kL;
    const long long t_ = row / parts;
    const int part = int(row - t_ * parts);
    const bool live = t_ < p.tokens;  // whole rows of lanes; the others keep the warp's shuffles complete
    const long long t = live ? t_ : p.tokens - 1;
    pdl_wait();
    pdl_launch_dependents();

    int pos = p.positions[t];
    if (pos < 0 || pos >= p.max_pos) {
        if (p.err && live) atomicOr(p.err, SANTA_ERR_POSITION);
        pos = pos < 0 ? 0 : p.max_pos - 1;
    }
    long long slot = p.slot_map ? p.slot_map[t] : t;
    if (slot >= p.total_tokens) {
        if (p.err && live) atomicOr(p.err, SANTA_ERR_SLOT);
        slot = -1;
    }
    const int half = p.rot_dim / 2;
    const float *cs = p.cos_sin + (size_t)pos * p.rot_dim;
    const bool turns = 8 * l < p.rot_dim;  // rot_dim is a multiple of 16: all of the lane's elements or none
    float c[8], s[8];  // of the lane's elements
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = 8 * l + j;
        const int f = p.interleaved ? i / 2 : (i < half ? i : i - half);
        c[j] = turns ? __ldg(cs + f) : 1.f;
        s[j] = turns ? __ldg(cs + half + f) : 0.f;
        if (p.interleaved ? (j & 1) == 0 : i < half) s[j] = -s[j];  // the first of a pair: a c - b s
    }
    // the lane that holds the other elements of the lane's pairs
    const int mate = p.interleaved || !turns ? l : (8 * l < half ? l + half / 8 : l - half / 8);
    const int mate_lane = (threadIdx.x & 31) - l + mate;

    const int rows = (p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (p.v ? p.Hkv : 0);
    for (int r0 = 0; r0 < rows; r0 += parts) {
        int r = r0 + part;
        const bool mine = live && r < rows;
        if (r >= rows) r = rows - 1;
        const T *src;
        T *dst;
        const void *weight = nullptr;
        bool turn = turns;
        int h = r;
        if (p.q && h < p.Hq) {
            src = static_cast<const T *>(p.q) + t * p.q_stride + h * D;
            dst = static_cast<T *>(p.q_out) + (t * p.Hq + h) * D;
            weight = p.q_weight;
        } else {
            if (p.q) h -= p.Hq;
            if (p.k && h < p.Hkv) {
                src = static_cast<const T *>(p.k) + t * p.k_stride + h * D;
                dst = slot < 0 ? nullptr : static_cast<T *>(p.k_cache) + (slot * p.Hkv + h) * D;
                weight = p.k_weight;
            } else {
                if (p.k) h -= p.Hkv;
                src = static_cast<const T *>(p.v) + t * p.v_stride + h * D;
                dst = slot < 0 ? nullptr : static_cast<T *>(p.v_cache) + (slot * p.Hkv + h) * D;
                turn = false;
            }
        }
        float x[8], y[8];
        Elems8<T>::load(src + 8 * l, x);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int o = 1; o < kL; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
        if (weight) {
            float w[8];
            Elems8<T>::load(static_cast<const T *>(weight) + 8 * l, w);
            const float inv = 1.f / sqrtf(ss / float(D) + p.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * inv * w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float other = __shfl_sync(kFull, x[j], mate_lane);
            if (p.interleaved) other = x[j ^ 1];
            y[j] = turn ? fmaf(x[j], c[j], other * s[j]) : x[j];
        }
        if (mine && dst) Elems8<T>::store(dst + 8 * l, y);
    }
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams &p, int dtype, int d, cudaStream_t stream) {
    const int rows = (p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (p.v ? p.Hkv : 0);
    int parts = 1;
    while (parts < rows && (long long)p.tokens * parts * (d / 8) < 152LL * 2048) parts *= 2;
    const long long threads = (long long)p.tokens * parts * (d / 8);
    const long long ctas = (threads + kRopeThreads - 1) / kRopeThreads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto go = [&](auto kern) {
        return launch_kernel(kern, dim3(unsigned(ctas)), dim3(kRopeThreads), 0, stream, true, 0, false, p, parts);
    };
    if (dtype == SANTA_BF16) return d == 128 ? go(norm_rope_kernel<uint16_t, 128>) : go(norm_rope_kernel<uint16_t, 64>);
    return d == 128 ? go(norm_rope_kernel<float, 128>) : go(norm_rope_kernel<float, 64>);
}

}  // namespace santa
