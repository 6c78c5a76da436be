// santa_window.cu -- exact decode attention over the visible keys (sliding window and
// sinks) of a bf16 or fp32 cache, contiguous or paged.
//
//   out = sum_j softmax(q . k_j / sqrt d) v_j over the keys j < sinks or j >= L - window,
// as one pass with a running maximum per query head of the group: with a block's logits
// x_j and M' = max(M, max_j x_j), e_j = 2^(x_j - M'),
//   Z' = Z 2^(M - M') + sum_j e_j,  O' = O 2^(M - M') + sum_j e_j v_j     (x in base 2).
// How the blocks of 32 keys are shared out and the pieces joined: santa_split.cuh.
//
// Every warp streams its blocks by itself through one K and one V buffer, filled by TMA
// (boxes of 32 rows x 128 bytes, 128-byte swizzle; a page holds whole blocks): the next
// block's K is requested as soon as the logits are formed, its V as soon as the sums are.
// Keys of a block that the query must not see get weight 0, and their V rows are
// overwritten with zeros in shared memory before they are multiplied, because they may
// hold anything (0 x NaN).
//
// bf16: logits and sums on the tensor cores (mma m16n8k16; keys x heads, then dims x
// heads, the group's heads padded to 8).  e is split into three bf16 parts (24 bits; two
// leave 2^-17 per weight, which shows in the fp32 output), transposed in registers
// (movmatrix), and each block's sums start from zero and are added to O by an fp32 fma:
// the tensor cores' additions truncate, and a chain over thousands of keys would drift.
//
// Bound by memory where there is enough of it: 64 ragged sequences of 4096 to 32768 tokens,
// window 4096 and 4 sinks (1.07 GB of K and V), 173 us = 6.2 TB/s, 0.92 of the copy rate; 12
// warps with one K and one V buffer each keep 196 KB in flight per SM.  At d = 64 that is half as
// much, and 16 sequences of 16384 keys take 126 us, 0.62 of the copy rate.  One sequence (16.8 MB)
// takes 10.6 us, a chain of dependent steps: lengths and plan 1.7 us, first K 0.8, first V 0.8,
// weights and sums 0.8, the last warp 0.3, join within the CTA 1.6, count 1, parts 3 (device
// timestamps, which add up to 10.0).
// fp32: a lane forms the whole dot products of one key (rows read along the swizzle
// without bank conflicts), then owns d / 32 dimensions of the sums.
#include "santa_split.cuh"
#include "santa_stream.cuh"

namespace santa {

namespace {

// (x, y) as three bf16 pairs whose sum is (x, y) to 2^-24 relative.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&o)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        o[i] = *reinterpret_cast<const uint32_t *>(&h);
        x -= __low2float(h);
        y -= __high2float(h);
    }
}

// GT: query heads of the group, for the register arrays of the fp32 path (bf16: 8, padded).
template <typename T, int D, int GT>
struct WindowGeom {
    using Geo = TileGeom<T, D>;
    static constexpr int kBytes = Geo::kBoxes * kChunkBoxBytes;  // K (or V) rows of a block: 4, 8 or 16 KiB
    static constexpr int kWarps = kBytes > 8192 ? 6 : GT > 4 ? 10 : 12;
    // shared memory: [kWarps][2] buffers; first pieces [kWarps][GT][D]; fp32: weights
    // [kWarps][32][GT]; mbarriers; what the CTA shares
    static constexpr size_t kFirst = size_t(kWarps) * 2 * kBytes;
    static constexpr size_t kEs = kFirst + size_t(kWarps) * GT * D * 4;
    static constexpr size_t kBars = kEs + (sizeof(T) == 4 ? size_t(kWarps) * 32 * GT * 4 : 0);
    static constexpr size_t kShared = (kBars + size_t(kWarps) * 2 * 8 + 15) & ~size_t(15);
    static constexpr size_t kTotal = kShared + sizeof(SplitShared<kWarps>);
    static_assert(kTotal <= 227 * 1024, "shared memory");
    // after the walk the buffers hold a warp's last piece; the joined heads' coefficients
    // and partial sums take the room of the first pieces and of other buffers
    static_assert(size_t(GT) * D * 4 <= size_t(2) * kBytes, "a piece fits a warp's buffers");
    static_assert(size_t(kSplitCtaBound) * kMaxGroup * 4 + size_t(kWarps) * 32 * 16 <= kFirst, "room to join");
};

template <typename T, int D, int GT, bool kPaged>
__global__ void __launch_bounds__(WindowGeom<T, D, GT>::kWarps * 32, 1)
    window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ SplitParams sp) {
    using WG = WindowGeom<T, D, GT>;
    using Geo = TileGeom<T, D>;
    constexpr int NW = WG::kWarps, kE = D / 32;
    constexpr bool kMma = sizeof(T) == 2;
    const Params &p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = p.G;

    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *kbuf = smem + size_t(warp) * 2 * WG::kBytes, *vbuf = kbuf + WG::kBytes;
    float *first_piece = reinterpret_cast<float *>(smem + WG::kFirst);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + WG::kBars) + warp * 2;
    SplitShared<NW> &sh = *reinterpret_cast<SplitShared<NW> *>(smem + WG::kShared);

    if (lane < 2) {
        mbar_init(&bars[lane], 1);
        sh.u0[2 * warp + lane] = -1;
    }
    if (threadIdx.x == 0) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    fence_barrier_init();
    __syncwarp();
    // Behind the prefix kernel of the same call nothing that this kernel reads or writes is that
    // kernel's, and what came before has ended when that kernel lets this one start: it runs beside
    // it, on SMs that it leaves free, and only ends after it, so that the kernel behind this one
    // finds the work of both.
    if (!sp.beside) pdl_wait();
    pdl_launch_dependents();

    Walk w;
    const int any = plan_walk<NW, kPaged>(sp, sh, w);
    if (any < 0) {
        if (sp.beside) pdl_wait();
        return;
    }

    auto issue = [&](int which, int row, int kvh) {
        if (lane != 0) return;
        uint64_t *bar = &bars[which];
        if (row >= 0) {
            unsigned char *dst = which ? vbuf : kbuf;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bar, WG::kBytes);
#pragma unroll
            for (int bx = 0; bx < Geo::kBoxes; ++bx)
                tma_load_3d(dst + bx * kChunkBoxBytes, which ? &vmap : &kmap, bar, bx * Geo::kBoxElems, kvh, row);
        } else {
            mbar_arrive(bar);
        }
    };

    // state of the group's heads.  bf16: lane (g, t) keeps heads 2t, 2t + 1: M, its own keys'
    // share of Z, and O^T in m16n8 tiles: Ot[m][j], Ot[m][2 + j] = O[2t + j][16 m + g], [.. + 8].
    // fp32: every lane keeps M of all heads, its own key's share of Z, and d / 32 elements of O.
    float M[kMma ? 2 : GT], Z[kMma ? 2 : GT];
    float Ot[kMma ? D / 16 : 1][4], O[kMma ? 1 : GT][kE];
    auto reset = [&]() {
#pragma unroll
        for (int h = 0; h < (kMma ? 2 : GT); ++h) {
            M[h] = -INFINITY;
            Z[h] = 0.f;
        }
#pragma unroll
        for (int m = 0; m < (kMma ? D / 16 : 1); ++m) Ot[m][0] = Ot[m][1] = Ot[m][2] = Ot[m][3] = 0.f;
#pragma unroll
        for (int h = 0; h < (kMma ? 1 : GT); ++h)
#pragma unroll
            for (int e = 0; e < kE; ++e) O[h][e] = 0.f;
    };
    // Closes the state for `head`: final outputs (kind 0), or piece `slot` with its sums at o.
    auto close = [&](const Head &head, bool final, int slot, float *o) {
        if constexpr (kMma) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) Z[j] += __shfl_xor_sync(kFull, Z[j], x);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int h = 2 * t + j;
                if (h < G) {
                    float *dst = final ? p.out + (size_t(head.b) * p.Hq + head.kvh * G + h) * D : o + h * D;
                    const float f = !final ? 1.f : Z[j] == 0.f ? 0.f : 1.f / Z[j];
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        dst[16 * m + g] = Ot[m][j] * f;
                        dst[16 * m + 8 + g] = Ot[m][2 + j] * f;
                    }
                    if (g == 0) {
                        if (!final) {
                            sh.M[slot][h] = M[j];
                            sh.Z[slot][h] = Z[j];
                        } else if (sp.own_mz) {
                            sp.own_mz[size_t(head.b) * p.Hq + head.kvh * G + h] = make_float2(M[j], Z[j]);
                        }
                    }
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < GT; ++h)
                if (h < G) {
                    const float z = warp_sum(Z[h]);
                    float *dst = final ? p.out + (size_t(head.b) * p.Hq + head.kvh * G + h) * D : o + h * D;
                    const float f = !final ? 1.f : z == 0.f ? 0.f : 1.f / z;
#pragma unroll
                    for (int e = 0; e < kE; ++e) dst[lane * kE + e] = O[h][e] * f;
                    if (lane == 0) {
                        if (!final) {
                            sh.M[slot][h] = M[h];
                            sh.Z[slot][h] = z;
                        } else if (sp.own_mz) {
                            sp.own_mz[size_t(head.b) * p.Hq + head.kvh * G + h] = make_float2(M[h], z);
                        }
                    }
                }
        }
        if (!final && lane == 0) note_piece(sh, slot, head);
    };

    const float scale2 = p.scale * 1.4426950408889634f;  // logits in base 2
    bool failed = false, k_flying = true;  // k_flying: the K barrier's phase is still to complete
    if (any > 0) {
        int sel = w.sel;  // the head of the block being computed; w runs one block ahead
        unsigned seen = seen_bits(w);  // keys of the block that the query sees
        int row = w.row;
        issue(0, row, w.heads[sel].kvh);
        issue(1, row, w.heads[sel].kvh);
        uint32_t qf[kMma ? D / 16 : 1][2];
        uint32_t phK = 0, phV = 0;
        bool fresh = true;  // the state is empty and q not loaded
        reset();
        for (bool more = true; more;) {
            const int n = w.n, moved = next_unit<kPaged>(sp, w);
            more = moved > 0;
            const unsigned next_seen = more ? seen_bits(w) : 0u;
            const int b = w.heads[sel].b, kvh = w.heads[sel].kvh;
            if (fresh && kMma) {
                // lane (g, t): dimensions 16 ks + 2t, +1 and 16 ks + 2t + 8, +9 of head g
                const uint32_t *qh = reinterpret_cast<const uint32_t *>(
                    static_cast<const uint16_t *>(p.q) + (size_t(b) * p.Hq + kvh * G + min(g, G - 1)) * D);
#pragma unroll
                for (int ks = 0; ks < (kMma ? D / 16 : 1); ++ks) {
                    qf[ks][0] = g < G ? load(qh + 8 * ks + t) : 0u;
                    qf[ks][1] = g < G ? load(qh + 8 * ks + 4 + t) : 0u;
                }
            }
            fresh = false;
            if (!mbar_wait(&bars[0], phK)) {
                failed = true;
                break;
            }
            phK ^= 1u;
            float c[2][4];
            float x[GT];
            if (row >= 0) {
                if constexpr (kMma) {
                    chunk_logits_mma<D>(kbuf, qf, lane, c);
                } else {
                    const float *qh = static_cast<const float *>(p.q) + (size_t(b) * p.Hq + kvh * G) * D;
                    float2 acc[GT];
#pragma unroll
                    for (int h = 0; h < GT; ++h) acc[h] = make_float2(0.f, 0.f);
#pragma unroll 4
                    for (int v = 0; v < D / 4; ++v) {
                        const float4 k4 = *reinterpret_cast<const float4 *>(kbuf + (v >> 3) * kChunkBoxBytes + lane * 128 +
                                                                            (((v & 7) ^ (lane & 7)) << 4));
#pragma unroll
                        for (int h = 0; h < GT; ++h) {
                            const float4 q4 = load(reinterpret_cast<const float4 *>(qh + min(h, G - 1) * D) + v);
                            acc[h] = __ffma2_rn(make_float2(q4.x, q4.y), make_float2(k4.x, k4.y), acc[h]);
                            acc[h] = __ffma2_rn(make_float2(q4.z, q4.w), make_float2(k4.z, k4.w), acc[h]);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < GT; ++h) x[h] = acc[h].x + acc[h].y;
                }
            }
            __syncwarp();
            if (more) issue(0, w.row, w.heads[w.sel].kvh);  // the K buffer is free
            k_flying = more;

            uint32_t pf[3][4];  // weights, part by part: keys 8 o + 2t, + 1 of head g
            float sc[kMma ? 2 : GT];
            if (row >= 0) {
                if constexpr (kMma) {
                    float xv[2][4];
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        const bool in = seen >> (8 * o + g) & 1;
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            xv[j][o] = in ? c[o >> 1][(o & 1) * 2 + j] * scale2 : -INFINITY;
                    }
                    float e[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float m = fmaxf(fmaxf(xv[j][0], xv[j][1]), fmaxf(xv[j][2], xv[j][3]));
#pragma unroll
                        for (int s = 4; s < 32; s <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
                        m = fmaxf(M[j], m);
                        const float ref = m == -INFINITY ? 0.f : m;
                        sc[j] = ex2(M[j] - ref);
                        M[j] = m;
                        float z = 0.f;
#pragma unroll
                        for (int o = 0; o < 4; ++o) {
                            e[j][o] = ex2(xv[j][o] - ref);
                            z += e[j][o];
                        }
                        Z[j] = fmaf(Z[j], sc[j], z);
                    }
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        uint32_t part[3];
                        split3(e[0][o], e[1][o], part);
#pragma unroll
                        for (int i = 0; i < 3; ++i) pf[i][o] = transpose_8x8(part[i]);
                    }
                } else {
                    float *es = reinterpret_cast<float *>(smem + WG::kEs) + warp * 32 * GT;
                    const bool in = seen >> lane & 1;
#pragma unroll
                    for (int h = 0; h < GT; ++h) {
                        const float xh = in ? x[h] * scale2 : -INFINITY;
                        const float m = fmaxf(M[h], warp_max(xh)), ref = m == -INFINITY ? 0.f : m;
                        const float e = ex2(xh - ref);
                        sc[h] = ex2(M[h] - ref);
                        M[h] = m;
                        Z[h] = fmaf(Z[h], sc[h], e);
                        es[lane * GT + h] = e;
                    }
                }
            }
            __syncwarp();
            if (!mbar_wait(&bars[1], phV)) {
                failed = true;
                break;
            }
            phV ^= 1u;
            if (row >= 0) {
                if (seen != kFull) {  // rows that the query must not see: zeros
                    for (int i = lane; i < kBlock * Geo::kBoxes * 8; i += 32) {
                        const int r = (i >> 3) % kBlock, bx = (i >> 3) / kBlock;
                        if (!(seen >> r & 1))
                            *reinterpret_cast<uint4 *>(vbuf + bx * kChunkBoxBytes + r * 128 + (i & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();  // before the next copy into this buffer
                    __syncwarp();
                }
                if constexpr (kMma) {
                    const int mq = lane >> 3, mi = lane & 7;
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks) {
                            // matrix mq: keys 16 ks + 8 (mq / 2) + row, dims 16 m + 8 (mq % 2) ..
                            const int key = 16 * ks + 8 * (mq >> 1) + mi, dv = 2 * m + (mq & 1);
                            uint32_t a[4];
                            ldmatrix_x4_trans(a, vbuf + (dv >> 3) * kChunkBoxBytes + key * 128 +
                                                     (((dv & 7) ^ (key & 7)) << 4));
#pragma unroll
                            for (int i = 2; i >= 0; --i) {
                                const uint32_t b[2] = {pf[i][2 * ks], pf[i][2 * ks + 1]};
                                mma_bf16_16816(acc, a, b);
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            Ot[m][j] = fmaf(Ot[m][j], sc[j], acc[j]);
                            Ot[m][2 + j] = fmaf(Ot[m][2 + j], sc[j], acc[2 + j]);
                        }
                    }
                } else {
                    const float *es = reinterpret_cast<const float *>(smem + WG::kEs) + warp * 32 * GT;
#pragma unroll
                    for (int h = 0; h < GT; ++h)
#pragma unroll
                        for (int e = 0; e < kE; ++e) O[h][e] *= sc[h];
                    const int byte = lane * kE * 4;  // of a row: box, 16-byte vector, offset in it
                    const unsigned char *vl = vbuf + (byte >> 7) * kChunkBoxBytes + (byte & 15);
                    const int vec = (byte & 127) >> 4;
#pragma unroll 4
                    for (int r = 0; r < kBlock; ++r) {
                        const float *src = reinterpret_cast<const float *>(vl + r * 128 + ((vec ^ (r & 7)) << 4));
                        float v[kE];
#pragma unroll
                        for (int e = 0; e < kE; ++e) v[e] = src[e];
#pragma unroll
                        for (int h = 0; h < GT; ++h) {
                            const float wgt = es[r * GT + h];
#pragma unroll
                            for (int e = 0; e < kE; ++e) O[h][e] = fmaf(wgt, v[e], O[h][e]);
                        }
                    }
                }
            }
            __syncwarp();
            if (more) issue(1, w.row, w.heads[w.sel].kvh);  // the V buffer is free

            if (moved != 1) {  // the stretch leaves the head
                const Head head = w.heads[sel];
                if (head.began && n + 1 == head.nb)
                    close(head, true, 0, nullptr);
                else if (more)
                    close(head, false, 2 * warp, first_piece + size_t(warp) * GT * D);
                else  // nothing in flight any more: the buffers are free
                    close(head, false, 2 * warp + 1, reinterpret_cast<float *>(kbuf));
                reset();
                fresh = true;
                sel = w.sel;
            }
            seen = next_seen;
            row = w.row;
        }
        if (failed) {
            // SANTA_ERR_TIMEOUT, location code 4; wait, bounded, for the copies in flight
            if (lane == 0) {
                raise_flag(p, SANTA_ERR_TIMEOUT | (4u << 8));
                const long long t0 = clock64();
                while (k_flying && !mbar_try_wait(&bars[0], phK) && clock64() - t0 < kWaitCycles) {
                }
                while (!mbar_try_wait(&bars[1], phV) && clock64() - t0 < kWaitCycles) {
                }
            }
            __syncwarp();
        }
    }
    // the joined heads' coefficients lie in the warps' buffers, whose pieces are consumed by then
    float *room = reinterpret_cast<float *>(smem);
    join_pieces<NW, D>(
        sp, sh,
        [&](int slot) {
            return slot & 1 ? reinterpret_cast<const float *>(smem + size_t(slot >> 1) * 2 * WG::kBytes)
                            : const_cast<const float *>(first_piece) + size_t(slot >> 1) * GT * D;
        },
        room);
    if (sp.beside) pdl_wait();
}

// Tensor map of a [rows][Hkv][d] cache: boxes of 128 bytes of one head's row x 32 rows.
bool kv_map(CUtensorMap *map, const void *base, int dtype, const Params &p) {
    const int es = dtype == SANTA_BF16 ? 2 : 4;
    const cuuint64_t dims[3] = {cuuint64_t(p.D), cuuint64_t(p.Hkv), cuuint64_t(p.total_tokens)};
    const cuuint64_t strides[2] = {cuuint64_t(p.D) * es, cuuint64_t(p.Hkv) * p.D * es};
    const cuuint32_t box[3] = {cuuint32_t(128 / es), 1u, cuuint32_t(kBlock)};
    return cache_map(map, dtype == SANTA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, base,
                     dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename T, int D, int GT>
cudaError_t launch(const SplitParams &sp, int dtype, cudaStream_t stream, const Timing &tm) {
    CUtensorMap kmap, vmap;
    if (!kv_map(&kmap, sp.p.k, dtype, sp.p) || !kv_map(&vmap, sp.p.v, dtype, sp.p)) return cudaErrorUnknown;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int ctas = sms < kSplitCtaBound ? sms : kSplitCtaBound;
    using WG = WindowGeom<T, D, GT>;
    auto go = [&](auto kern) {
        cudaError_t r = ensure_smem(kern, WG::kTotal);
        if (r != cudaSuccess) return r;
        record_event(tm.begin, stream);
        r = launch_kernel(kern, dim3(unsigned(ctas)), dim3(WG::kWarps * 32), WG::kTotal, stream, true, 0, false, kmap, vmap,
                          sp);
        record_event(tm.end, stream);
        return r;
    };
    return sp.p.page_table ? go(window_kernel<T, D, GT, true>) : go(window_kernel<T, D, GT, false>);
}

template <typename T, int D>
cudaError_t launch_g(const SplitParams &sp, int dtype, cudaStream_t stream, const Timing &tm) {
    if constexpr (sizeof(T) == 2) {
        return sp.p.G <= 4 ? launch<T, D, 4>(sp, dtype, stream, tm) : launch<T, D, 8>(sp, dtype, stream, tm);
    } else {
        if (sp.p.G == 1) return launch<T, D, 1>(sp, dtype, stream, tm);
        if (sp.p.G == 2) return launch<T, D, 2>(sp, dtype, stream, tm);
        return sp.p.G <= 4 ? launch<T, D, 4>(sp, dtype, stream, tm) : launch<T, D, 8>(sp, dtype, stream, tm);
    }
}

}  // namespace

cudaError_t launch_window(const SplitParams &sp, int dtype, cudaStream_t stream, const Timing &tm) {
    if (dtype == SANTA_BF16)
        return sp.p.D == 128 ? launch_g<uint16_t, 128>(sp, dtype, stream, tm) : launch_g<uint16_t, 64>(sp, dtype, stream, tm);
    return sp.p.D == 128 ? launch_g<float, 128>(sp, dtype, stream, tm) : launch_g<float, 64>(sp, dtype, stream, tm);
}

}  // namespace santa
