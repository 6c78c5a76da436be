// santa_weights.cu -- the attention weight that each cached key receives, added to its score.
//
// Pass 1 of prop leaves, per query head and chunk c of 32 keys, the record (m_c, z_c) and the
// stash e_i = exp(x_i - m_c).  With M = max_c m_c and Z = sum_c z_c exp(m_c - M) the weight of
// key i is A_i = e_i exp(m_c - M) / Z, so the scores cost a read of the records and the stash
// (4 bytes per key and query head, still in L2), not another one of K:
//   score' = decay * score + sum over the group's heads of A_i.
// The chunks of a (sequence, KV head) are cut over CTAs, `per` each; a CTA forms (M, Z) of the group's
// heads from all their records (a record per 32 keys: a sixteenth of the stash), then the factors
// exp(m_c - M) / Z of its own chunks, and its warps take the chunks, a lane per key, kAhead in flight.
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kWeightThreads = 256;
constexpr int kWeightWarps = kWeightThreads / 32;

__device__ __forceinline__ float rec_m(unsigned long long r) { return __uint_as_float(unsigned(r)); }
__device__ __forceinline__ float rec_z(unsigned long long r) { return __uint_as_float(unsigned(r >> 32)); }

// (m, z) joined with (m2, z2).
__device__ __forceinline__ void join(float &m, float &z, float m2, float z2) {
    const float n = fmaxf(m, m2), ref = n == -INFINITY ? 0.f : n;
    z = z * expf(m - ref) + z2 * expf(m2 - ref);
    m = n;
}

constexpr int kMaxPer = 128;  // chunks of a CTA, at most

template <int G, bool kPaged>
__global__ void __launch_bounds__(kWeightThreads, G == 8 ? 3 : 4)
    key_weights_kernel(const __grid_constant__ WeightParams w, int per) {
    constexpr int kPer = kWeightWarps / G;     // warps per head while (M, Z) are formed
    constexpr int kAhead = G == 8 ? 2 : 4;     // chunks of a warp in flight
    const Params &p = w.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.y, b = blockIdx.z;
    __shared__ float sm[kWeightWarps], sz[kWeightWarps];
    __shared__ float M[G], inv[G], factor[kMaxPer * G];
    long long start;
    const int L = seq_bounds<kPaged>(p, b, &start);
    const int n = (L + 31) / 32, c0 = blockIdx.x * per, c1 = min(n, c0 + per);
    if (c0 >= c1) return;
    const unsigned long long *rec = p.rec + (size_t(b) * p.Hq + kvh * G) * p.nch;
    {
        constexpr int kRec = 8;  // records of a lane in flight
        const unsigned long long *r = rec + size_t(warp / kPer) * p.nch;
        float m = -INFINITY, z = 0.f;
        for (int c = (warp % kPer) * 32 + lane; c < n; c += kRec * 32 * kPer) {
            unsigned long long v[kRec];
#pragma unroll
            for (int u = 0; u < kRec; ++u) {
                const int i = c + u * 32 * kPer;
                v[u] = i < n ? r[i] : 0xff800000ull;  // (-inf, 0)
            }
            float top = rec_m(v[0]);
#pragma unroll
            for (int u = 1; u < kRec; ++u) top = fmaxf(top, rec_m(v[u]));
            const float ref = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < kRec; ++u) sum = fmaf(rec_z(v[u]), expf(rec_m(v[u]) - ref), sum);
            join(m, z, top, sum);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) join(m, z, __shfl_xor_sync(kFull, m, o), __shfl_xor_sync(kFull, z, o));
        if (lane == 0) {
            sm[warp] = m;
            sz[warp] = z;
        }
    }
    __syncthreads();
    if (threadIdx.x < G) {
        float m = sm[threadIdx.x * kPer], z = sz[threadIdx.x * kPer];
        for (int i = 1; i < kPer; ++i) join(m, z, sm[threadIdx.x * kPer + i], sz[threadIdx.x * kPer + i]);
        M[threadIdx.x] = m == -INFINITY ? 0.f : m;
        inv[threadIdx.x] = z == 0.f ? 0.f : 1.f / z;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (c1 - c0) * G; i += kWeightThreads) {
        const int g = i % G, c = i / G;
        factor[i] = expf(rec_m(rec[size_t(g) * p.nch + c0 + c]) - M[g]) * inv[g];
    }
    __syncthreads();
    const float *stash = p.stash + (size_t(b) * p.Hq + kvh * G) * p.nch * 32 + lane;
    const size_t plane = size_t(kvh) * p.total_tokens;
    for (int c = c0 + warp; c < c1; c += kWeightWarps * kAhead) {
        float e[kAhead][G], old[kAhead];
        long long row[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int ch = c + u * kWeightWarps, key = ch * 32 + lane;
            const bool in = ch < c1 && key < L;
            row[u] = in ? key_row<kPaged>(p, b, start, key) : -1;
#pragma unroll
            for (int g = 0; g < G; ++g) e[u][g] = in ? stash[(size_t(g) * p.nch + ch) * 32] : 0.f;
            old[u] = row[u] >= 0 && w.scores && key < L - w.fresh ? w.scores[plane + row[u]] * w.decay : 0.f;
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (row[u] < 0) continue;
            const float *f = factor + (c + u * kWeightWarps - c0) * G;
            float a = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) a += f[g] == 0.f ? 0.f : e[u][g] * f[g];  // a chunk without mass may have no stash
            w.scores_out[plane + row[u]] = old[u] + a;
        }
    }
}

}  // namespace

cudaError_t launch_key_weights(const WeightParams &w, cudaStream_t stream) {
    const Params &p = w.p;
    // as many chunks per CTA (every CTA reads all records of its heads) as leave four CTAs per SM
    const long long chunks = (long long)p.B * p.Hkv * p.nch;
    int per = kMaxPer;
    while (per > 4 * kWeightWarps && chunks / per < 4 * 152) per /= 2;
    const dim3 grid(unsigned((p.nch + per - 1) / per), unsigned(p.Hkv), unsigned(p.B));
    auto go = [&](auto kern) { return launch_kernel(kern, grid, dim3(kWeightThreads), 0, stream, false, 0, false, w, per); };
    auto pick = [&](auto paged) {
        constexpr bool kP = decltype(paged)::value;
        switch (p.G) {
            case 1: return go(key_weights_kernel<1, kP>);
            case 2: return go(key_weights_kernel<2, kP>);
            case 4: return go(key_weights_kernel<4, kP>);
            case 8: return go(key_weights_kernel<8, kP>);
            default: return cudaErrorNotSupported;
        }
    };
    return p.page_table ? pick(std::true_type()) : pick(std::false_type());
}

}  // namespace santa
