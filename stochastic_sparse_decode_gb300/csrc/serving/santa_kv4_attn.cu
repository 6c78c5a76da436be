// santa_kv4_attn.cu -- exact decode attention over a K/V cache held in 4 bits.
//
// A key row stands for k_i = m_g + s_g n_i (codes n_i in 0 .. 15; scale s_g and minimum m_g
// of element i's group g), a value row likewise, so
//   q . k_j     = sum_g s_jg (q_g . n_jg) + m_jg sum(q_g)
//   sum_j e_j v_j = sum_j (e_j s_jg) n_j  + sum_j e_j m_jg          (group by group),
// and both large products run on the tensor cores (fp16 mma m16n8k16) on the codes as
// they lie in memory.  A code needs no conversion: masked out of its word it is, as an fp16
// bit pattern, the subnormal n 2^-24 (low nibble of a byte) or n 2^-20 (high nibble), which
// the tensor cores multiply exactly; the powers of two go into q and the final factor.
// One 32-bit word of K gives a lane the A fragments of two products (4 ands, 1 shift); a
// word of V, paired with the next key's by byte permutes, those of four (2 permutes, 8
// ands, 2 shifts), so nothing is staged through shared memory: codes go from global
// memory to registers, the next block's while the current one is computed.
//
// Precision: q is scaled by a power of two per head to fit fp16 (a bf16 q is exact so; an
// fp32 q is taken in two parts, 22 bits), the weights e_j s_jg in two parts (22 bits) under
// a running power of two that keeps the largest scale of the row's values in range;
// everything else is fp32.  The online softmax and the sharing out of the keys are those
// of the windowed kernel (santa_split.cuh): each block's sums start from zero and join O
// by an fp32 fma.
#include <cuda_fp16.h>

#include "santa_split.cuh"

namespace santa {

namespace {

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (x, y) as an fp16 pair, and what the rounding left.
__device__ __forceinline__ uint32_t half_pair(float &x, float &y) {
    const __half2 h = __floats2half2_rn(x, y);
    x -= __low2float(h);
    y -= __high2float(h);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 half_values(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }
// Exponent of |x|, held to +-100 (0 gives -100).
__device__ __forceinline__ int exponent(float x) {
    const int e = int((__float_as_uint(x) >> 23) & 255u) - 127;
    return e < -100 ? -100 : e > 100 ? 100 : e;
}

constexpr uint32_t kLo = 0x000f000fu, kHi = 0x00f000f0u;

template <int D, int GT>
struct Kv4Geom {
    static constexpr int kWarps = 12;
    static constexpr size_t kPieces = size_t(kWarps) * 2 * GT * D * 4;  // first and last pieces
    static constexpr size_t kTotal = kPieces + sizeof(SplitShared<kWarps>);
    static_assert(size_t(kSplitCtaBound) * GT * 4 + size_t(kWarps) * 32 * 16 <= kPieces, "room to join");
    static_assert(kTotal <= 227 * 1024, "shared memory");
};

// What a lane (g = lane / 4, t = lane % 4) loads of a block of 32 records.
template <int D>
struct Block4 {
    static constexpr int kW = D / 32;  // words of K's codes per key and lane; V: kW / 2
    static constexpr int kG = D / 64;
    uint32_t k[4][kW];          // keys 8 o + g: words kW t ..
    uint32_t v[4][2][kW / 2];   // keys 8 o + 2t + i: words kW / 2 g ..
    uint32_t par[2 * kG];       // key `lane`: (scale, minimum) of K's groups, then V's
};

template <int D, typename Q, int GT, bool kPaged>
__global__ void __launch_bounds__(Kv4Geom<D, GT>::kWarps * 32, 1) kv4_kernel(const __grid_constant__ SplitParams sp) {
    using Geom = Kv4Geom<D, GT>;
    using Blk = Block4<D>;
    constexpr int NW = Geom::kWarps, kW = Blk::kW, kG = Blk::kG, kTiles = D / 16;
    constexpr int kQ = sizeof(Q) == 2 ? 1 : 2;  // fp16 parts of q
    constexpr int kRec = kv4_record(D);
    const Params &p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = p.G;
    extern __shared__ __align__(16) unsigned char smem[];
    float *pieces = reinterpret_cast<float *>(smem);  // [warp][first, last][GT][D]
    SplitShared<NW> &sh = *reinterpret_cast<SplitShared<NW> *>(smem + Geom::kPieces);
    if (lane < 2) sh.u0[2 * warp + lane] = -1;
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();

    Walk w;
    const bool any = plan_walk<NW, kPaged>(sp, sh, w);
    if ((int)blockIdx.x >= w.ctas) return;

    const uint32_t step = uint32_t(p.Hkv) * kRec;  // bytes from a key's record to the next key's
    Blk blk;
    // Record of the first key of block n of head h, null for a bad page (its keys are dropped).
    auto block_at = [&](const Head &h, int key0) -> const unsigned char * {
        const long long row = key_row<kPaged>(p, h.b, h.start, key0);
        return row < 0 ? nullptr : sp.kv4 + ((size_t)row * p.Hkv + h.kvh) * kRec;
    };
    // which keys of the block at key0 the query sees, a bit each
    auto seen_bits = [&](const Head &h, int key0, const unsigned char *rec) {
        const int key = key0 + lane;
        return __ballot_sync(kFull, rec && key < h.vis.L && (key < h.vis.s || key >= h.vis.lo));
    };
    auto load_k = [&](const unsigned char *rec, unsigned seen) {
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            const int r = 8 * o + g;
            const unsigned char *src = rec + r * step + t * (kW * 4);
            if constexpr (kW == 4) {
                const uint4 x = seen >> r & 1 ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
                blk.k[o][0] = x.x, blk.k[o][1] = x.y, blk.k[o][2] = x.z, blk.k[o][3] = x.w;
            } else {
                const uint2 x = seen >> r & 1 ? __ldg(reinterpret_cast<const uint2 *>(src)) : make_uint2(0, 0);
                blk.k[o][0] = x.x, blk.k[o][1] = x.y;
            }
        }
    };
    auto load_v = [&](const unsigned char *rec, unsigned seen) {
#pragma unroll
        for (int o = 0; o < 4; ++o)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 8 * o + 2 * t + i;
                const unsigned char *src = rec + r * step + D / 2 + g * (kW * 2);
                if constexpr (kW == 4) {
                    const uint2 x = seen >> r & 1 ? __ldg(reinterpret_cast<const uint2 *>(src)) : make_uint2(0, 0);
                    blk.v[o][i][0] = x.x, blk.v[o][i][1] = x.y;
                } else {
                    blk.v[o][i][0] = seen >> r & 1 ? __ldg(reinterpret_cast<const uint32_t *>(src)) : 0u;
                }
            }
    };
    auto load_par = [&](const unsigned char *rec, unsigned seen) {
        const unsigned char *src = rec + lane * step + D;
        if constexpr (kG == 2) {
            const uint4 x = seen >> lane & 1 ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0, 0, 0, 0);
            blk.par[0] = x.x, blk.par[1] = x.y, blk.par[2] = x.z, blk.par[3] = x.w;
        } else {
            const uint2 x = seen >> lane & 1 ? __ldg(reinterpret_cast<const uint2 *>(src)) : make_uint2(0, 0);
            blk.par[0] = x.x, blk.par[1] = x.y;
        }
    };

    // State of heads 2t, 2t + 1: M, the lane's own keys' share of Z and of the sums of
    // e_j m_jg, and O^T: tile (word i of the lane's V words, q) holds elements 2q (Ot[..][j])
    // and 2q + 1 (Ot[..][2 + j]) of word (kW / 2) g + i, times fscale 2^-24 and 2^-20.
    float M[2], Z[2], base[kG][2], Ot[kTiles][4], fscale;
    auto reset = [&]() {
        M[0] = M[1] = -INFINITY;
        Z[0] = Z[1] = 0.f;
        fscale = pow2(60);  // larger than any block allows
#pragma unroll
        for (int i = 0; i < kG; ++i) base[i][0] = base[i][1] = 0.f;
#pragma unroll
        for (int m = 0; m < kTiles; ++m) Ot[m][0] = Ot[m][1] = Ot[m][2] = Ot[m][3] = 0.f;
    };
    auto close = [&](const Head &head, bool final, int slot) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                Z[j] += __shfl_xor_sync(kFull, Z[j], x);
#pragma unroll
                for (int i = 0; i < kG; ++i) base[i][j] += __shfl_xor_sync(kFull, base[i][j], x);
            }
        const float f = 1.f / fscale;  // a power of two
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = 2 * t + j;
            if (h < G) {
                float *dst = final ? p.out + (size_t(head.b) * p.Hq + head.kvh * G + h) * D
                                   : pieces + (size_t(slot) * GT + h) * D;
                const float inv = !final ? 1.f : Z[j] == 0.f ? 0.f : 1.f / Z[j];
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    const int i = m / 4, at = 8 * (kW / 2 * g + i) + 2 * (m % 4);
                    *reinterpret_cast<float2 *>(dst + at) =
                        make_float2(fmaf(Ot[m][j], f * 16777216.f, base[i % kG][j]) * inv,
                                    fmaf(Ot[m][2 + j], f * 1048576.f, base[i % kG][j]) * inv);
                }
                if (!final && g == 0) {
                    sh.M[slot][h] = M[j];
                    sh.Z[slot][h] = Z[j];
                }
            }
        }
        if (!final && lane == 0) note_piece(sh, slot, head);
    };

    if (any) {
        Head head = w.head;  // of the block being computed; w runs one block ahead
        const unsigned char *rec = block_at(head, head.first_key(w.n));
        unsigned seen = seen_bits(head, head.first_key(w.n), rec);
        load_k(rec, seen);
        load_par(rec, seen);
        load_v(rec, seen);
        const long long x_first = w.x;
        uint32_t qf[kQ][kW][2][2];  // [part][word][step]: elements (0, 4), (1, 5) / 16, then (2, 6), (3, 7) / 16
        float qsum[kG][2], kq[2];   // of heads 2t, 2t + 1: sum(q_g), and the factor of the products; base 2
        bool fresh = true;
        reset();
        for (bool more = true; more;) {
            more = next_unit<kPaged>(sp, w);
            const bool same = more && w.head.u0 == head.u0;
            const unsigned char *next = nullptr;
            unsigned next_seen = 0;
            if (more) {
                next = block_at(w.head, w.head.first_key(w.n));
                next_seen = seen_bits(w.head, w.head.first_key(w.n), next);
            }
            if (fresh) {
                fresh = false;
                // this lane's kW words (8 elements each) of head g
                const Q *qh = static_cast<const Q *>(p.q) + (size_t(head.b) * p.Hq + head.kvh * G + min(g, G - 1)) * D +
                              t * kW * 8;
                float x[kW][8], mx = 0.f, sum[kG];
#pragma unroll
                for (int i = 0; i < kG; ++i) sum[i] = 0.f;
#pragma unroll
                for (int u = 0; u < kW; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[u][i] = g < G ? to_float<Q>(__ldg(qh + 8 * u + i)) : 0.f;
                        mx = fmaxf(mx, fabsf(x[u][i]));
                        sum[u % kG] += x[u][i];
                    }
#pragma unroll
                for (int s = 1; s < 4; s <<= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, s));
#pragma unroll
                    for (int i = 0; i < kG; ++i) sum[i] += __shfl_xor_sync(kFull, sum[i], s);
                }
                const int e = exponent(mx);
                const float f = pow2(14 - e);
#pragma unroll
                for (int u = 0; u < kW; ++u)
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi) {
                            float a = x[u][2 * s + hi] * f, b = x[u][2 * s + hi + 4] * f;
                            if (hi) {
                                a *= 0.0625f;
                                b *= 0.0625f;
                            }
#pragma unroll
                            for (int i = 0; i < kQ; ++i) qf[i][u][s][hi] = half_pair(a, b);
                        }
                const float scale2 = p.scale * 1.4426950408889634f;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int src = 4 * (2 * t + j);
                    kq[j] = pow2(__shfl_sync(kFull, e, src) + 10) * scale2;  // 2^24 2^(e - 14)
#pragma unroll
                    for (int i = 0; i < kG; ++i) qsum[i][j] = __shfl_sync(kFull, sum[i], src) * scale2;
                }
            }

            // ---- q . n of the block, group by group: c[mt][group], keys 16 mt + g and + 8
            float c[2][kG][4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                for (int i = 0; i < kG; ++i) c[mt][i][0] = c[mt][i][1] = c[mt][i][2] = c[mt][i][3] = 0.f;
#pragma unroll
                for (int u = 0; u < kW; ++u)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const uint32_t a = blk.k[2 * mt][u] >> (8 * s), b = blk.k[2 * mt + 1][u] >> (8 * s);
                        const uint32_t frag[4] = {a & kLo, b & kLo, a & kHi, b & kHi};
#pragma unroll
                        for (int i = kQ - 1; i >= 0; --i)
                            mma_f16_16816(c[mt][u % kG], frag, qf[i][u][s][0], qf[i][u][s][1]);
                    }
            }
            if (more) load_k(next, next_seen);

            // ---- online softmax; the weights times the values' scales, as B fragments
            uint32_t pf[kG][2][4];  // [group][part][octet]
            float sc[2];
            {
                float e[2][4];
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    const int r = 8 * o + g;
                    float y[2] = {0.f, 0.f}, z[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < kG; ++i) {
                        const float2 sm = half_values(__shfl_sync(kFull, blk.par[i], r));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            y[j] = fmaf(sm.x, c[o >> 1][i][(o & 1) * 2 + j], y[j]);
                            z[j] = fmaf(sm.y, qsum[i][j], z[j]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) e[j][o] = seen >> r & 1 ? fmaf(y[j], kq[j], z[j]) : -INFINITY;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float m = fmaxf(fmaxf(e[j][0], e[j][1]), fmaxf(e[j][2], e[j][3]));
#pragma unroll
                    for (int s = 4; s < 32; s <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
                    m = fmaxf(M[j], m);
                    const float ref = m == -INFINITY ? 0.f : m;
                    sc[j] = ex2(M[j] - ref);
                    M[j] = m;
                    float z = 0.f;
#pragma unroll
                    for (int o = 0; o < 4; ++o) {
                        e[j][o] = ex2(e[j][o] - ref);
                        z += e[j][o];
                    }
                    Z[j] = fmaf(Z[j], sc[j], z);
#pragma unroll
                    for (int i = 0; i < kG; ++i) base[i][j] *= sc[j];
                }
                // the largest scale of the block's values decides the power of two
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < kG; ++i) top = fmaxf(top, fabsf(half_values(blk.par[kG + i]).x));
                top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
                if (top * fscale >= 32768.f) {
                    const float lower = pow2(14 - exponent(top)), ratio = lower / fscale;
                    sc[0] *= ratio;
                    sc[1] *= ratio;
                    fscale = lower;
                }
#pragma unroll
                for (int o = 0; o < 4; ++o)
#pragma unroll
                    for (int i = 0; i < kG; ++i) {
                        const float2 sm = half_values(__shfl_sync(kFull, blk.par[kG + i], 8 * o + g));
                        const float s = sm.x * fscale;
                        float a = e[0][o] * s, b = e[1][o] * s;
#pragma unroll
                        for (int part = 0; part < 2; ++part) pf[i][part][o] = transpose_8x8(half_pair(a, b));
                        base[i][0] = fmaf(e[0][o], sm.y, base[i][0]);
                        base[i][1] = fmaf(e[1][o], sm.y, base[i][1]);
                    }
            }
            if (more) load_par(next, next_seen);

            // ---- O += (e s) n, tile by tile
#pragma unroll
            for (int i = 0; i < kW / 2; ++i) {
                // pairs of keys: low and high halves of the word, octet by octet
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    lo[o] = __byte_perm(blk.v[o][0][i], blk.v[o][1][i], 0x5410);
                    hi[o] = __byte_perm(blk.v[o][0][i], blk.v[o][1][i], 0x7632);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int sh8 = (q & 1) * 8;
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) {
                        const uint32_t a = (q < 2 ? lo : hi)[2 * ks] >> sh8, b = (q < 2 ? lo : hi)[2 * ks + 1] >> sh8;
                        const uint32_t frag[4] = {a & kLo, a & kHi, b & kLo, b & kHi};
#pragma unroll
                        for (int part = 1; part >= 0; --part)
                            mma_f16_16816(acc, frag, pf[i % kG][part][2 * ks], pf[i % kG][part][2 * ks + 1]);
                    }
                    float(&o)[4] = Ot[4 * i + q];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        o[j] = fmaf(o[j], sc[j], acc[j]);
                        o[2 + j] = fmaf(o[2 + j], sc[j], acc[2 + j]);
                    }
                }
            }
            if (more) load_v(next, next_seen);

            if (!same) {  // the stretch leaves the head
                const bool whole = head.u0 >= x_first && head.u0 + head.nb <= w.x_end;
                close(head, whole, 2 * warp + (more ? 0 : 1));
                reset();
                fresh = true;
                head = w.head;
            }
            seen = next_seen;
        }
    }
    float *room = reinterpret_cast<float *>(smem);  // the pieces are consumed when it is written
    join_pieces<NW, D>(
        sp, sh, w, [&](int slot) { return const_cast<const float *>(pieces) + size_t(slot) * GT * D; }, room,
        room + kSplitCtaBound * GT);
}

template <int D, typename Q, int GT>
cudaError_t launch(const SplitParams &sp, cudaStream_t stream, const Timing &tm) {
    using Geom = Kv4Geom<D, GT>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int ctas = sms < kSplitCtaBound ? sms : kSplitCtaBound;
    auto go = [&](auto kern) {
        cudaError_t r = ensure_smem(kern, Geom::kTotal);
        if (r != cudaSuccess) return r;
        record_event(tm.begin, stream);
        r = launch_kernel(kern, dim3(unsigned(ctas)), dim3(Geom::kWarps * 32), Geom::kTotal, stream, true, 0, false, sp);
        record_event(tm.end, stream);
        return r;
    };
    return sp.p.page_table ? go(kv4_kernel<D, Q, GT, true>) : go(kv4_kernel<D, Q, GT, false>);
}

template <int D, typename Q>
cudaError_t launch_g(const SplitParams &sp, cudaStream_t stream, const Timing &tm) {
    return sp.p.G <= 4 ? launch<D, Q, 4>(sp, stream, tm) : launch<D, Q, 8>(sp, stream, tm);
}

}  // namespace

cudaError_t launch_kv4(const SplitParams &sp, int dtype, cudaStream_t stream, const Timing &tm) {
    if (dtype == SANTA_BF16)
        return sp.p.D == 128 ? launch_g<128, uint16_t>(sp, stream, tm) : launch_g<64, uint16_t>(sp, stream, tm);
    return sp.p.D == 128 ? launch_g<128, float>(sp, stream, tm) : launch_g<64, float>(sp, stream, tm);
}

}  // namespace santa
