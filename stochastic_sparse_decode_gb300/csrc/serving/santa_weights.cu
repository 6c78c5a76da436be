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
//
// Pass 1 itself (key_logits_kernel, bf16, batches): prop's walk passes by the chunks that a sequence
// of max_len would have and this one has not, which costs a ragged batch a quarter of its time.
// Here the blocks that there are are shared out equally (santa_split.cuh), each warp streaming its
// stretch through two buffers; per chunk the arithmetic, and so every bit, is prop's.
//
// Bound by memory: 16 sequences of 4096 to 32768 keys, 32 query and 8 KV heads of 128 (604 MB of K, 38 MB
// of stash), 110 us = 5.8 TB/s, 0.88 of the copy rate (prop's walk 134); the scores 17 us more, of which
// the stash read back and 19 MB of scores would be 9.  One sequence of 32768: 13.5 and 4.9 us.
#include "santa_split.cuh"
#include "santa_stream.cuh"

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
    __shared__ int first_row[kMaxPer];  // of each of the CTA's chunks (a chunk lies on one page); -1: a bad page
    long long start;
    const int L = seq_bounds<kPaged>(p, b, &start);
    const int n = (L + 31) / 32, c0 = blockIdx.x * per, c1 = min(n, c0 + per);
    if (c0 >= c1) return;
    for (int c = threadIdx.x; c < c1 - c0; c += kWeightThreads)
        first_row[c] = int(key_row<kPaged>(p, b, start, (c0 + c) * 32));
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
        int row[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int ch = c + u * kWeightWarps, key = ch * 32 + lane;
            const bool in = ch < c1 && key < L;
            row[u] = in ? first_row[ch - c0] : -1;
            if (row[u] >= 0) row[u] += lane;
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

template <int D>
struct LogitGeom {
    using Geo = TileGeom<uint16_t, D>;
    static constexpr int kWarps = D == 128 ? 12 : 16;
    static constexpr int kBytes = Geo::kBoxes * kChunkBoxBytes;  // keys of a block
    static constexpr size_t kBars = size_t(kWarps) * 2 * kBytes, kShared = kBars + size_t(kWarps) * 2 * 8;
    static constexpr size_t kTotal = kShared + sizeof(SplitShared<kWarps>);
    static_assert(kTotal <= 227 * 1024, "shared memory");
};

template <int D, int G, bool kPaged>
__global__ void __launch_bounds__(LogitGeom<D>::kWarps * 32, 1)
    key_logits_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ SplitParams sp) {
    using LG = LogitGeom<D>;
    using Geo = TileGeom<uint16_t, D>;
    constexpr int NW = LG::kWarps;
    const Params &p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *buf = smem + size_t(warp) * 2 * LG::kBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + LG::kBars) + warp * 2;
    SplitShared<NW> &sh = *reinterpret_cast<SplitShared<NW> *>(smem + LG::kShared);
    if (lane < 2) mbar_init(&bars[lane], 1);
    if (threadIdx.x == 0) prefetch_tensormap(&kmap);
    fence_barrier_init();
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();
    Walk w;
    if (plan_walk<NW, kPaged>(sp, sh, w) <= 0) return;
    auto issue = [&](int slot, int row, int kvh) {
        if (lane != 0) return;
        if (row >= 0) {
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&bars[slot], LG::kBytes);
#pragma unroll
            for (int bx = 0; bx < Geo::kBoxes; ++bx)
                tma_load_3d_hint(buf + slot * LG::kBytes + bx * kChunkBoxBytes, &kmap, &bars[slot], bx * Geo::kBoxElems, kvh,
                                 row, l2_evict_first());
        } else {
            mbar_arrive(&bars[slot]);
        }
    };
    issue(0, w.row, w.heads[w.sel].kvh);
    uint32_t qf[D / 16][2];
    int qb = -1, qkvh = -1;
    bool failed = false, more = true;
    int i = 0;
    for (; more; ++i) {
        const int slot = i & 1, b = w.heads[w.sel].b, kvh = w.heads[w.sel].kvh, ch = w.key0 / kBlock, row = w.row;
        const int len = min(kBlock, w.heads[w.sel].vis.L - w.key0);
        more = next_unit<kPaged>(sp, w) > 0;
        if (more) issue(slot ^ 1, w.row, w.heads[w.sel].kvh);
        if (b != qb || kvh != qkvh) {
            load_q_frag<D, G>(p, b, kvh * G, lane, qf);
            qb = b;
            qkvh = kvh;
        }
        if (!mbar_wait(&bars[slot], (i >> 1) & 1)) {
            failed = true;
            break;
        }
        float xv[2][4], m[2], z[2];
        if (row >= 0) {
            float c[2][4];
            chunk_logits_mma<D>(buf + slot * LG::kBytes, qf, lane, c);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    xv[j][k] = 8 * k + g < len ? c[k >> 1][(k & 1) * 2 + j] * p.scale : -INFINITY;
                m[j] = fmaxf(fmaxf(xv[j][0], xv[j][1]), fmaxf(xv[j][2], xv[j][3]));
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int j = 0; j < 2; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(kFull, m[j], o));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                z[j] = 0.f;
#pragma unroll
                for (int k = 3; k >= 0; --k) {
                    xv[j][k] = __expf(xv[j][k] - m[j]);  // 0 for keys past the end
                    z[j] += xv[j][k];
                }
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                for (int j = 0; j < 2; ++j) z[j] += __shfl_xor_sync(kFull, z[j], o);
        } else {  // a bad page id (flagged): the chunk carries no mass
            m[0] = m[1] = -INFINITY;
            z[0] = z[1] = 0.f;
        }
        __syncwarp();  // the buffer is free for the walk's unit after the next
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 2 * t + j;
            if (h >= G) continue;
            const size_t at = (size_t(b) * p.Hq + kvh * G + h) * p.nch + ch;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (row >= 0 && 8 * k + g < len) p.stash[at * kChunkRows + 8 * k + g] = xv[j][k];
            if (g == 0) store_record(p.rec + at, m[j], z[j]);
        }
    }
    if (failed && lane == 0) {  // location code 6; wait, bounded, for the copies in flight
        raise_flag(p, SANTA_ERR_TIMEOUT | (6u << 8));
        const long long t0 = clock64();
        for (int k = i; k <= i + (more ? 1 : 0); ++k)
            while (!mbar_try_wait(&bars[k & 1], (k >> 1) & 1) && clock64() - t0 < kWaitCycles) {
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

cudaError_t launch_key_logits(const SplitParams &sp, const CUtensorMap &kmap, cudaStream_t stream, const Timing &tm) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    record_event(tm.begin, stream);
    auto go = [&](auto kern, int warps, size_t smem) {
        const cudaError_t r = ensure_smem(kern, smem);
        if (r != cudaSuccess) return r;
        return launch_kernel(kern, dim3(unsigned(sms)), dim3(warps * 32), smem, stream, true, 0, false, kmap, sp);
    };
    auto pick_d = [&](auto group, auto paged) {
        constexpr int kG = decltype(group)::value;
        constexpr bool kP = decltype(paged)::value;
        return sp.p.D == 128 ? go(key_logits_kernel<128, kG, kP>, LogitGeom<128>::kWarps, LogitGeom<128>::kTotal)
                             : go(key_logits_kernel<64, kG, kP>, LogitGeom<64>::kWarps, LogitGeom<64>::kTotal);
    };
    auto pick = [&](auto group) {
        return sp.p.page_table ? pick_d(group, std::true_type()) : pick_d(group, std::false_type());
    };
    switch (sp.p.G) {
        case 1: e = pick(std::integral_constant<int, 1>()); break;
        case 2: e = pick(std::integral_constant<int, 2>()); break;
        case 4: e = pick(std::integral_constant<int, 4>()); break;
        case 8: e = pick(std::integral_constant<int, 8>()); break;
        default: e = cudaErrorNotSupported;
    }
    record_event(tm.end, stream);
    return e;
}

}  // namespace santa
