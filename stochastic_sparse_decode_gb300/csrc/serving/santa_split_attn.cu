// santa_split_attn.cu -- decode attention over the visible keys (window + sinks), on a
// 16-bit, 32-bit or 4-bit cache: the plain form of the kernel.
//
// One CTA per (KV head, sequence); its warps take the visible keys in turn, a lane
// holding D / 32 elements of the row, and keep an online softmax (M, Z, O) per query head
// of the group: M' = max(M, x), Z' = Z exp(M - M') + exp(x - M'), O' likewise.  The
// warps' states are joined in order at the end.
#include <cuda_fp16.h>

#include "santa_visible.cuh"

namespace santa {

namespace {

constexpr int kWarps = 8;

struct Kv4Elem {};  // tag: a 4-bit cache

// A lane's D / 32 elements of K (which = 0) or V (1) of a cache row.
template <typename C, int D>
__device__ __forceinline__ void load_row(const SplitParams &sp, int which, long long row, int kvh, int lane,
                                         float (&x)[D / 32]) {
    if constexpr (sizeof(C) > 1) {
        const C *src = static_cast<const C *>(which ? sp.p.v : sp.p.k) + ((size_t)row * sp.p.Hkv + kvh) * D;
        RowSlice<C, D> r;
        r.load(src, lane);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = r.v[e];
    } else {
        const unsigned char *rec = sp.kv4 + ((size_t)row * sp.p.Hkv + kvh) * kv4_record(D);
        const int i = lane * (D / 32), g = (i / 8) % (D / 64);
        uint32_t w;
        if constexpr (D == 128)
            w = *reinterpret_cast<const uint16_t *>(rec + which * 64 + lane * 2);
        else
            w = rec[which * 32 + lane];
        const float2 sm = __half22float2(reinterpret_cast<const __half2 *>(rec + D + which * (D / 16))[g]);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) x[e] = fmaf(sm.x, float((w >> (4 * e)) & 15u), sm.y);
    }
}

template <typename C, typename Q, int D, bool kPaged>
__global__ void __launch_bounds__(kWarps * 32) attend_kernel(const SplitParams sp) {
    constexpr int kE = D / 32;
    const Params &p = sp.p;
    const int kvh = blockIdx.x, b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float s_m[kWarps][kMaxGroup], s_z[kWarps][kMaxGroup], s_o[kWarps][kMaxGroup][D];
    long long start;
    const int L = seq_bounds<kPaged>(p, b, &start);
    const Visible vis = visible(L, sp.window, sp.sinks);
    float q[kMaxGroup][kE], O[kMaxGroup][kE], M[kMaxGroup], Z[kMaxGroup];
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
        M[h] = -INFINITY;
        Z[h] = 0.f;
        RowSlice<Q, D> r;
        if (h < p.G) r.load(static_cast<const Q *>(p.q) + ((size_t)b * p.Hq + kvh * p.G + h) * D, lane);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
            q[h][e] = h < p.G ? r.v[e] : 0.f;
            O[h][e] = 0.f;
        }
    }
    for (int j = warp; j < vis.count(); j += kWarps) {
        const long long row = key_row<kPaged>(p, b, start, vis.key(j));
        if (row < 0) continue;  // bad page id (flagged): its keys are dropped
        float k[kE], v[kE];
        load_row<C, D>(sp, 0, row, kvh, lane, k);
        load_row<C, D>(sp, 1, row, kvh, lane, v);
#pragma unroll
        for (int h = 0; h < kMaxGroup; ++h) {
            if (h >= p.G) break;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < kE; ++e) x = fmaf(q[h][e], k[e], x);
            x = warp_sum(x) * p.scale;
            const float m = fmaxf(M[h], x), sc = expf(M[h] - m), w = expf(x - m);
            M[h] = m;
            Z[h] = fmaf(Z[h], sc, w);
#pragma unroll
            for (int e = 0; e < kE; ++e) O[h][e] = fmaf(O[h][e], sc, w * v[e]);
        }
    }
#pragma unroll
    for (int h = 0; h < kMaxGroup; ++h) {
        if (lane == 0) {
            s_m[warp][h] = M[h];
            s_z[warp][h] = Z[h];
        }
#pragma unroll
        for (int e = 0; e < kE; ++e) s_o[warp][h][lane * kE + e] = O[h][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.G * D; i += kWarps * 32) {
        const int h = i / D, e = i % D;
        float m = -INFINITY, z = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w][h]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float c = s_z[w][h] == 0.f ? 0.f : expf(s_m[w][h] - m);
            z = fmaf(s_z[w][h], c, z);
            o = fmaf(s_o[w][h][e], c, o);
        }
        p.out[((size_t)b * p.Hq + kvh * p.G + h) * D + e] = z == 0.f ? 0.f : o / z;
    }
}

template <typename C, typename Q>
cudaError_t launch(const SplitParams &sp, cudaStream_t stream, const Timing &tm) {
    const Params &p = sp.p;
    auto go = [&](auto kern) {
        record_event(tm.begin, stream);
        const cudaError_t e = launch_kernel(kern, dim3(p.Hkv, p.B), dim3(kWarps * 32), 0, stream, false, 0, false, sp);
        record_event(tm.end, stream);
        return e;
    };
    if (p.page_table) return p.D == 128 ? go(attend_kernel<C, Q, 128, true>) : go(attend_kernel<C, Q, 64, true>);
    return p.D == 128 ? go(attend_kernel<C, Q, 128, false>) : go(attend_kernel<C, Q, 64, false>);
}

}  // namespace

cudaError_t launch_kv4(const SplitParams &sp, int dtype, cudaStream_t stream, const Timing &tm) {
    return dtype == SANTA_BF16 ? launch<Kv4Elem, uint16_t>(sp, stream, tm) : launch<Kv4Elem, float>(sp, stream, tm);
}

}  // namespace santa
