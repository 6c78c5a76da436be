// santa_kv4_attn.cu -- exact decode attention over a K/V cache held in 4 bits.
//
// A key row stands for k_i = m_g + s_g n_i (codes n_i in 0 .. 15; scale s_g and minimum m_g
// of element i's group g), a value row likewise, so that group by group
//   q . k_j       = sum_g s_jg (q_g . n_jg)       + m_jg sum(q_g)
//   sum_j e_j v_j = sum_j (e_j s_jg) (n_j - 8)    + sum_j e_j (m_jg + 8 s_jg)
// and both large products run on the tensor cores (fp16 mma m16n8k16).
//
// K's codes need no conversion: shifted to bits 4 .. 7 and masked out of its word a code is,
// as an fp16 bit pattern, the subnormal n 2^-20; the power of two goes into the logits'
// factor.  V's codes are centred, two by one LOP3 (masked onto the low bits of 1024) and one
// exact add (1024 + n - 1032, or 1024 + 16 n - 1152).  The centring is not for looks: with n
// itself the two terms of the second line are each about 2.6 standard deviations of the values
// and cancel to the mean of thousands of them, and what the tensor cores truncate showed as
// 3e-4 of the output at 32768 keys, all the more as subnormals (products are aligned by their
// operands' exponents, which a subnormal's value may lie far below).  Errors of the logits are
// independent from key to key and average out; low nibbles left at bits 0 .. 3 (n 2^-24), two
// shifts less per word, cost up to 1.2e-6 of the output of a few keys.
//
// Codes are the A operand of both (rows: keys, then elements), queries and weights the B
// operand (columns: heads).  A word of K's codes gives a lane the A fragments of two products
// (3 shifts, 4 ands); two keys' words of V, paired by byte permutes, those of eight.  The
// weights turn from the layout in which the logits come out into the one in which they go in
// by movmatrix.
//
// Precision: q is scaled by a power of two per head to fit fp16 (a bf16 q is exact so; an
// fp32 q is taken in two parts, 22 bits); the weights e_j s_jg likewise in two parts, under a
// running power of two that keeps the largest scale of the row's values in range.  With at
// most four heads the eight columns hold the heads twice: the logits of the copies cost
// nothing, and the copies' weights are the second parts, so one product takes both.
// Everything else is fp32.  The online softmax and the sharing out of the keys are those of
// the windowed kernel (santa_split.cuh): each block's sums start from zero and join O by an
// fp32 fma.
//
// The rows' scales and minima are converted once, by the lane that has the key, and shared
// through shared memory, each twice in a row for packed fp32 arithmetic on pairs of heads.
// d = 128: a warp's blocks come by TMA (boxes of 32 records) into two buffers of its own.
// d = 64: a record is 72 bytes, which TMA's strides cannot express; the codes go from global
// memory to registers, the next block's while the current one is computed.
//
// Bound by instructions: about 800 per warp and block of 32 keys, 0.58 issued per cycle and
// scheduler by 4 warps of 128 registers (which d = 128 with up to four heads in bf16 exceeds: 88
// bytes of spill stores, 68 paged).  16 sequences of 32768 tokens, 32 query and 8 KV heads of 128
// (604 MB): 138 us = 4.4 TB/s, 0.64 of the copy rate (the same walk without arithmetic: 98 us).  On
// the way, for the 16: one warp per key in fp32 4612 us; tensor cores on converted registers 199; q
// and the weights as the A operand 197; codes as the A operand with the heads twice 132, centred
// 155, one LOP3 per pair 147, K as subnormals 138.  12 warps of 168 registers: 218 us at the 132
// step; so are the shapes that 16 warps do not fit, five to eight heads (shared memory) 216 us and
// fp32 queries (registers of their second part, and its products) 212.  d = 64: 96 us for half the
// bytes, as scales, softmax and weights are work per key.  1000 sequences of 100 keys: 74 us, work
// per head (four units each).
// One sequence of 32768 (22.2 us): lengths and plan 1.7 us, the first blocks of all warps, 11 MB
// at once, 4, three or four blocks a warp 8, join within the CTA 2.2, count 1, parts 5 (device
// timestamps).
#include <cuda_fp16.h>

#include "santa_split.cuh"
#include "santa_stream.cuh"

namespace santa {

namespace {

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same on a zero accumulator.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// (x, y) as an fp16 pair; x and y become what the rounding left.
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

// (w & mask) | 0x6400 twice: codes on top of 1024 in fp16, whose last bits count ones.  As PTX,
// because the compiler spends two instructions on the expression (128 more per block).
template <uint32_t kMask>
__device__ __forceinline__ uint32_t on_1024(uint32_t w) {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w), "n"(kMask), "r"(0x64006400u));
    return x;
}
__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;  // nibbles of bytes 0 and 2
// The low nibbles of bytes 0 and 2 of w less 8, as an fp16 pair; the high nibbles less 8, times 16.
__device__ __forceinline__ uint32_t low_codes(uint32_t w) { return add_half2(on_1024<kLow>(w), 0xe408e408u); }
__device__ __forceinline__ uint32_t high_codes(uint32_t w) { return add_half2(on_1024<kHigh>(w), 0xe480e480u); }

template <int D, typename Q, int GT>
struct Kv4Geom {
    static constexpr bool kTma = D == 128;
    static constexpr int kQ = sizeof(Q) == 2 ? 1 : 2;        // fp16 parts of q
    static constexpr int kWarps = kTma && (GT > 4 || kQ > 1) ? 12 : 16;
    static constexpr bool kTwice = GT <= 4;                  // the columns hold the heads twice
    static constexpr int kG = D / 64;
    static constexpr int kBuf = kTma ? kBlock * kv4_record(D) : 0;  // bytes of a block
    static constexpr int kParBytes = kBlock * kG * 32;       // its scales and minima of K and of V, each twice, fp32
    static constexpr size_t kPiece = size_t(GT) * D * 4;
    // shared memory: two buffers per warp (its last piece when the walk is over; d = 64: that piece
    // alone), first pieces, parameters, mbarriers, shared state
    static constexpr size_t kSlot = kTma ? 2 * size_t(kBuf) : kPiece;
    static constexpr size_t kFirst = kWarps * kSlot;
    static constexpr size_t kParOff = kFirst + kWarps * kPiece;
    static constexpr size_t kBars = kParOff + size_t(kWarps) * kParBytes;
    static constexpr size_t kShared = kBars + size_t(kWarps) * 16;
    static constexpr size_t kTotal = kShared + sizeof(SplitShared<kWarps>);
    static_assert(kPiece <= kSlot && kSlot % 128 == 0, "a piece fits a warp's buffers");
    static_assert(size_t(kSplitCtaBound) * kMaxGroup * 4 + size_t(kWarps) * 32 * 16 <= kBars, "room to join");
    static_assert(kTotal <= 227 * 1024, "shared memory");
};

template <int D, typename Q, int GT, bool kPaged>
__global__ void __launch_bounds__(Kv4Geom<D, Q, GT>::kWarps * 32, 1)
    kv4_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ SplitParams sp) {
    using Geom = Kv4Geom<D, Q, GT>;
    constexpr int NW = Geom::kWarps, kG = Geom::kG, kQ = Geom::kQ;
    constexpr bool kTma = Geom::kTma;
    constexpr int kW = D / 32;   // words of K's codes per key and lane; V: kW / 2
    constexpr int kTiles = D / 16;
    constexpr bool kTwice = Geom::kTwice;
    constexpr int kParts = kTwice ? 1 : 2;  // products that take the weights' parts
    constexpr int kRec = kv4_record(D);
    const Params &p = sp.p;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int G = p.G;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *buf = smem + warp * Geom::kSlot;
    float *first_piece = reinterpret_cast<float *>(smem + Geom::kFirst);                    // [warp][GT][D]
    float4 *par = reinterpret_cast<float4 *>(smem + Geom::kParOff + warp * Geom::kParBytes);  // see below
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Geom::kBars) + warp * 2;
    SplitShared<NW> &sh = *reinterpret_cast<SplitShared<NW> *>(smem + Geom::kShared);
    if (lane < 2) {
        sh.u0[2 * warp + lane] = -1;
        if (kTma) mbar_init(&bars[lane], 1);
    }
    if (kTma) {
        if (threadIdx.x == 0) prefetch_tensormap(&map);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();

    Walk w;
    const int any = plan_walk<NW, kPaged>(sp, sh, w);
    if (any < 0) return;

    // d = 128: starts the copy of the walk's block into buffer i (a dropped block completes the
    // buffer's phase with a plain arrive)
    auto issue = [&](int i) {
        if (lane != 0) return;
        if (w.row >= 0) {
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&bars[i], Geom::kBuf);
            tma_load_3d(buf + i * Geom::kBuf, &map, &bars[i], 0, w.heads[w.sel].kvh, w.row);
        } else {
            mbar_arrive(&bars[i]);
        }
    };
    // the block's codes: K of keys 8 o + g (words kW t ..), V of keys 8 o + 2t + i (words kW / 2 g ..),
    // and key `lane`'s pairs (scale, minimum): K's groups, then V's.  d = 64: from global memory,
    // zeros for keys that the query must not see (rec: the block's first record).
    const uint32_t step = kTma ? kRec : uint32_t(p.Hkv) * kRec;  // bytes from a key's record to the next key's
    uint32_t kc[4][kW], vc[4][2][kW / 2], pc[2 * kG];
    auto record = [&]() { return sp.kv4 + ((size_t)(w.row < 0 ? 0 : w.row) * p.Hkv + w.heads[w.sel].kvh) * kRec; };
    auto load_k = [&](const unsigned char *rec, unsigned seen) {
        const unsigned char *src = rec + g * step + t * (kW * 4);
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            if constexpr (kTma) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src);
                kc[o][0] = x.x, kc[o][1] = x.y, kc[o][kW - 2] = x.z, kc[o][kW - 1] = x.w;
            } else {
                const uint2 x = seen >> (8 * o + g) & 1 ? load(reinterpret_cast<const uint2 *>(src)) : make_uint2(0, 0);
                kc[o][0] = x.x, kc[o][1] = x.y;
            }
            src += 8 * step;
        }
    };
    auto load_v = [&](const unsigned char *rec, unsigned seen) {
        const unsigned char *src = rec + 2 * t * step + D / 2 + g * (kW * 2);
#pragma unroll
        for (int o = 0; o < 4; ++o) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const unsigned char *at = src + i * step;
                if constexpr (kTma) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(at);
                    vc[o][i][0] = x.x, vc[o][i][kW / 2 - 1] = x.y;
                } else {
                    vc[o][i][0] = seen >> (8 * o + 2 * t + i) & 1 ? load(reinterpret_cast<const uint32_t *>(at)) : 0u;
                }
            }
            src += 8 * step;
        }
    };
    auto load_par = [&](const unsigned char *rec, unsigned seen) {
        const unsigned char *src = rec + lane * step + D;
        const bool in = seen >> lane & 1;  // the others' scales may be anything
        if constexpr (kTma) {
            const uint4 x = in ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
            pc[0] = x.x, pc[1] = x.y, pc[2 * kG - 2] = x.z, pc[2 * kG - 1] = x.w;
        } else {
            const uint2 x = in ? load(reinterpret_cast<const uint2 *>(src)) : make_uint2(0, 0);
            pc[0] = x.x, pc[1] = x.y;
        }
    };

    // State of the heads of columns 2t, 2t + 1: M, the shares of the lane's own keys of Z and of
    // the sums of e_j (m + 8 s), and O^T: tile (word i of the lane's V words, q) holds elements 2q
    // (O[..][0 .. 1]) and 2q + 1 (O[..][2 .. 3]) of word (kW / 2) g + i, times fscale and 16 fscale.
    const int h0 = kTwice ? 2 * (t & 1) : 2 * t;  // head of column 2t
    float M[2], Z[2], base[kG][2], O[kTiles][4], fscale;
    auto reset = [&]() {
        M[0] = M[1] = -INFINITY;
        Z[0] = Z[1] = 0.f;
        fscale = pow2(60);  // larger than any block allows
#pragma unroll
        for (int i = 0; i < kG; ++i) base[i][0] = base[i][1] = 0.f;
#pragma unroll
        for (int n = 0; n < kTiles; ++n) O[n][0] = O[n][1] = O[n][2] = O[n][3] = 0.f;
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
        if constexpr (kTwice) {  // the two parts' sums
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) O[n][j] += __shfl_xor_sync(kFull, O[n][j], 2);
        }
        const float f0 = 1.f / fscale, f1 = 0.0625f / fscale;  // powers of two
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int h = h0 + j;
            if (h < G && (!kTwice || t < 2)) {
                float *dst = final ? p.out + (size_t(head.b) * p.Hq + head.kvh * G + h) * D
                                   : (slot & 1 ? reinterpret_cast<float *>(buf) : first_piece + size_t(warp) * GT * D) + h * D;
                const float inv = !final ? 1.f : Z[j] == 0.f ? 0.f : 1.f / Z[j];
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    const int i = n / 4, at = 8 * (kW / 2 * g + i) + 2 * (n % 4);
                    *reinterpret_cast<float2 *>(dst + at) = make_float2(fmaf(O[n][j], f0, base[i % kG][j]) * inv,
                                                                        fmaf(O[n][2 + j], f1, base[i % kG][j]) * inv);
                }
                if (!final && g == 0) {
                    sh.M[slot][h] = M[j];
                    sh.Z[slot][h] = Z[j];
                }
            }
        }
        if (!final && lane == 0) note_piece(sh, slot, head);
    };

    if (any > 0) {
        int sel = w.sel;  // the head of the block being computed; w runs one block ahead
        unsigned seen = seen_bits(w);
        if constexpr (kTma) {
            issue(0);
        } else {
            const unsigned char *rec = record();
            load_par(rec, seen);
            load_k(rec, seen);
            load_v(rec, seen);
        }
        uint32_t qf[kQ][kW][4];  // the B operand of q, see below
        int cur = 0;             // the buffer of the block
        uint32_t phase = 0;
        float2 qsum[kG], kq;     // of the columns' heads: sum(q_g) and the logits' factor: x = kq y, base 2
        const float part2 = kTwice && t >= 2 ? 1.f : 0.f;
        bool fresh = true, failed = false;
        reset();
        for (bool more = true; more;) {
            const int n = w.n, moved = next_unit<kPaged>(sp, w);
            more = moved > 0;
            const unsigned char *next = nullptr;
            unsigned next_seen = 0;
            if (more) {
                next_seen = seen_bits(w);
                if constexpr (!kTma) next = record();
            }
            if (fresh) {
                fresh = false;
                // q as the B operand: word u's step s takes elements (2s, 2s + 4) and (2s + 1, 2s + 5) of
                // words kW t + u of the head of column g
                const int hg = kTwice ? g & 3 : g;
                const Q *qh = static_cast<const Q *>(p.q) +
                              (size_t(w.heads[sel].b) * p.Hq + w.heads[sel].kvh * G + min(hg, G - 1)) * D + t * kW * 8;
                float x[kW][8], mx = 0.f, sum[kG];
#pragma unroll
                for (int i = 0; i < kG; ++i) sum[i] = 0.f;
#pragma unroll
                for (int u = 0; u < kW; ++u) {
                    constexpr int kVec = 8 * sizeof(Q) / 16;
#pragma unroll
                    for (int i = 0; i < kVec; ++i) {
                        float2 pr[Vec16<Q>::kPairs];
                        Vec16<Q>::unpack(load(reinterpret_cast<const uint4 *>(qh + 8 * u) + i), pr);
#pragma unroll
                        for (int j = 0; j < Vec16<Q>::kPairs; ++j) {
                            x[u][2 * (i * Vec16<Q>::kPairs + j)] = pr[j].x;
                            x[u][2 * (i * Vec16<Q>::kPairs + j) + 1] = pr[j].y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (hg >= G) x[u][i] = 0.f;
                        mx = fmaxf(mx, fabsf(x[u][i]));
                        sum[u % kG] += x[u][i];
                    }
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
                for (int u = 0; u < kW; ++u) {
                    float a[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = x[u][i] * f;
#pragma unroll
                    for (int part = 0; part < kQ; ++part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) qf[part][u][i] = half_pair(a[i], a[i + 4]);
                }
                // y = sum_g s_g c_g + m_g sum(q_g) / (2^20 2^(e - 14)), in the products' units
                const int e0 = __shfl_sync(kFull, e, 4 * h0), e1 = __shfl_sync(kFull, e, 4 * (h0 + 1));
                const float scale2 = p.scale * 1.4426950408889634f;
                kq = make_float2(pow2(e0 + 6) * scale2, pow2(e1 + 6) * scale2);
#pragma unroll
                for (int i = 0; i < kG; ++i)
                    qsum[i] = make_float2(__shfl_sync(kFull, sum[i], 4 * h0) * pow2(-6 - e0),
                                          __shfl_sync(kFull, sum[i], 4 * (h0 + 1)) * pow2(-6 - e1));
            }
            if constexpr (kTma) {
                if (!mbar_wait(&bars[cur], phase >> cur & 1)) {
                    failed = true;
                    break;
                }
                phase ^= 1u << cur;
                // the next block's buffer was read by the block before this one, which every lane is
                // past.  Not before this block has landed: its copy would share the memory with the
                // first blocks of all warps.
                if (more) issue(cur ^ 1);
                load_par(buf + cur * Geom::kBuf, seen);
                load_k(buf + cur * Geom::kBuf, seen);
            }

            // ---- key `lane`'s scales and minima, in fp32, V's scales times the running power of two
            float lower = 1.f;
            {
                float2 sm[2 * kG];
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < 2 * kG; ++i) sm[i] = half_values(pc[i]);
#pragma unroll
                for (int i = 0; i < kG; ++i) top = fmaxf(top, fabsf(sm[kG + i].x));
                top = __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(top)));
                if (top * fscale >= 32768.f) {
                    const float f = pow2(14 - exponent(top));
                    lower = f / fscale;
                    fscale = f;
                }
                if (!kTma && more) load_par(next, next_seen);
                // per key and group (s, s, m, m) of K, then (s, s, m + 8 s, m + 8 s) of V; the slots of a
                // key turn with the key against bank conflicts
#pragma unroll
                for (int i = 0; i < 2 * kG; ++i) {
                    const float sc = i < kG ? sm[i].x : sm[i].x * fscale;
                    const float mid = i < kG ? sm[i].y : fmaf(8.f, sm[i].x, sm[i].y);  // V: m + 8 s
                    par[lane * 2 * kG + ((i + lane) & (2 * kG - 1))] = make_float4(sc, sc, mid, mid);
                }
                __syncwarp();
            }
            auto params = [&](int i, int r, float2 &sc, float2 &mn) {  // i: group of K, kG + group of V
                const float4 v = par[r * 2 * kG + ((i + r) & (2 * kG - 1))];
                sc = make_float2(v.x, v.y);
                mn = make_float2(v.z, v.w);
            };

            // ---- logits of the columns' heads and keys 8 o + g
            float2 y[4];
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                float c[kG][4];
#pragma unroll
                for (int u = 0; u < kW; ++u)
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        // nibbles 2s (and 2s + 4), then 2s + 1 (and 2s + 5), each at bits 4 .. 7
                        const uint32_t ka = kc[2 * mt][u], kb = kc[2 * mt + 1][u];
                        const uint32_t a0 = (s ? ka >> 4 : ka << 4) & kHigh, a1 = (s ? ka >> 8 : ka) & kHigh;
                        const uint32_t b0 = (s ? kb >> 4 : kb << 4) & kHigh, b1 = (s ? kb >> 8 : kb) & kHigh;
#pragma unroll
                        for (int part = kQ - 1; part >= 0; --part) {
                            if (u < kG && s == 0 && part == kQ - 1)
                                mma_f16_zero(c[u % kG], a0, b0, a1, b1, qf[part][u][2 * s],
                                             qf[part][u][2 * s + 1]);
                            else
                                mma_f16(c[u % kG], a0, b0, a1, b1, qf[part][u][2 * s],
                                        qf[part][u][2 * s + 1]);
                        }
                    }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int o = 2 * mt + hf;
                    float2 sc, mn;
                    params(0, 8 * o + g, sc, mn);
                    y[o] = __ffma2_rn(sc, make_float2(c[0][2 * hf], c[0][2 * hf + 1]), __fmul2_rn(mn, qsum[0]));
                    if constexpr (kG == 2) {
                        params(1, 8 * o + g, sc, mn);
                        y[o] = __ffma2_rn(mn, qsum[1], y[o]);
                        y[o] = __ffma2_rn(sc, make_float2(c[1][2 * hf], c[1][2 * hf + 1]), y[o]);
                    }
                }
            }

            // ---- online softmax
            if (seen != kFull) {
#pragma unroll
                for (int o = 0; o < 4; ++o)
                    if (!(seen >> (8 * o + g) & 1)) y[o] = make_float2(-INFINITY, -INFINITY);
            }
            float2 sc;
            {
                float m0 = fmaxf(fmaxf(y[0].x, y[1].x), fmaxf(y[2].x, y[3].x));
                float m1 = fmaxf(fmaxf(y[0].y, y[1].y), fmaxf(y[2].y, y[3].y));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    m0 = fmaxf(m0, __shfl_xor_sync(kFull, m0, x));
                    m1 = fmaxf(m1, __shfl_xor_sync(kFull, m1, x));
                }
                m0 = fmaxf(M[0], m0 * kq.x);
                m1 = fmaxf(M[1], m1 * kq.y);
                const float2 ref = make_float2(m0 == -INFINITY ? 0.f : -m0, m1 == -INFINITY ? 0.f : -m1);
                sc = make_float2(ex2(M[0] + ref.x), ex2(M[1] + ref.y));
                M[0] = m0;
                M[1] = m1;
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    y[o] = __ffma2_rn(y[o], kq, ref);
                    y[o] = make_float2(ex2(y[o].x), ex2(y[o].y));
                }
                const float2 z = __fadd2_rn(__fadd2_rn(y[0], y[1]), __fadd2_rn(y[2], y[3]));
                const float2 zz = __ffma2_rn(make_float2(Z[0], Z[1]), sc, z);
                Z[0] = zz.x;
                Z[1] = zz.y;
            }

            // ---- the weights times V's scales, as the B operand
            uint32_t pf[kG][kParts][4];  // [group][part][octet]
#pragma unroll
            for (int i = 0; i < kG; ++i) {
                float2 bs = __fmul2_rn(make_float2(base[i][0], base[i][1]), sc);
#pragma unroll
                for (int o = 0; o < 4; ++o) {
                    float2 s, mn;
                    params(kG + i, 8 * o + g, s, mn);
                    bs = __ffma2_rn(y[o], mn, bs);
                    const float2 v = __fmul2_rn(y[o], s);
                    const __half2 h = __floats2half2_rn(v.x, v.y);
                    if constexpr (kTwice) {  // first parts in columns 0 .. 3, what they leave in 4 .. 7
                        const __half2 l = __floats2half2_rn(fmaf(-part2, __low2float(h), v.x), fmaf(-part2, __high2float(h), v.y));
                        pf[i][0][o] = transpose_8x8(*reinterpret_cast<const uint32_t *>(&l));
                    } else {
                        const __half2 l = __floats2half2_rn(v.x - __low2float(h), v.y - __high2float(h));
                        pf[i][0][o] = transpose_8x8(*reinterpret_cast<const uint32_t *>(&h));
                        pf[i][kParts - 1][o] = transpose_8x8(*reinterpret_cast<const uint32_t *>(&l));
                    }
                }
                base[i][0] = bs.x;
                base[i][1] = bs.y;
            }
            __syncwarp();  // the parameters are read: the next block's may be written
            if (!kTma && more) load_k(next, next_seen);
            if constexpr (kTma) load_v(buf + cur * Geom::kBuf, seen);

            // ---- O += (e s) n, tile by tile
            const float2 sco = make_float2(sc.x * lower, sc.y * lower);
#pragma unroll
            for (int i = 0; i < kW / 2; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t pr[4];  // 4 nibbles of keys 8 o + 2t (low half) and + 1 (high half)
#pragma unroll
                    for (int o = 0; o < 4; ++o) pr[o] = __byte_perm(vc[o][0][i], vc[o][1][i], half ? 0x7632 : 0x5410);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (s)
#pragma unroll
                            for (int o = 0; o < 4; ++o) pr[o] >>= 8;
                        float acc[4];
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                            for (int part = kParts - 1; part >= 0; --part) {
                                const uint32_t(&b)[4] = pf[i % kG][part];
                                const uint32_t a = pr[2 * ks], c = pr[2 * ks + 1];
                                if (ks == 0 && part == kParts - 1)
                                    mma_f16_zero(acc, low_codes(a), high_codes(a), low_codes(c), high_codes(c), b[2 * ks],
                                                 b[2 * ks + 1]);
                                else
                                    mma_f16(acc, low_codes(a), high_codes(a), low_codes(c), high_codes(c), b[2 * ks],
                                            b[2 * ks + 1]);
                            }
                        float(&o)[4] = O[4 * i + 2 * half + s];
                        const float2 lo = __ffma2_rn(make_float2(o[0], o[1]), sco, make_float2(acc[0], acc[1]));
                        const float2 hi = __ffma2_rn(make_float2(o[2], o[3]), sco, make_float2(acc[2], acc[3]));
                        o[0] = lo.x, o[1] = lo.y, o[2] = hi.x, o[3] = hi.y;
                    }
                }
            if (!kTma && more) load_v(next, next_seen);
            cur ^= 1;

            if (moved != 1) {  // the stretch leaves the head
                const Head head = w.heads[sel];
                close(head, head.began && n + 1 == head.nb, 2 * warp + (more ? 0 : 1));
                reset();
                fresh = true;
                sel = w.sel;
            }
            seen = next_seen;
        }
        if (failed) {
            // SANTA_ERR_TIMEOUT, location code 5; wait, bounded, for the copies in flight
            if (lane == 0) {
                raise_flag(p, SANTA_ERR_TIMEOUT | (5u << 8));
                const long long t0 = clock64();
                while (!mbar_try_wait(&bars[cur], phase >> cur & 1) && clock64() - t0 < kWaitCycles) {
                }
            }
            __syncwarp();
        }
    }
    join_pieces<NW, D>(
        sp, sh,
        [&](int slot) {
            return slot & 1 ? reinterpret_cast<const float *>(smem + (slot >> 1) * Geom::kSlot)
                            : const_cast<const float *>(first_piece) + size_t(slot >> 1) * GT * D;
        },
        reinterpret_cast<float *>(smem));  // the pieces are consumed when it is written
}

template <int D, typename Q, int GT>
cudaError_t launch(const SplitParams &sp, cudaStream_t stream, const Timing &tm) {
    using Geom = Kv4Geom<D, Q, GT>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int ctas = sms < kSplitCtaBound ? sms : kSplitCtaBound;
    CUtensorMap map = {};
    if (Geom::kTma) {  // [rows][Hkv][record], boxes of one head's record x 32 rows
        const cuuint64_t dims[3] = {cuuint64_t(kv4_record(D)), cuuint64_t(sp.p.Hkv), cuuint64_t(sp.p.total_tokens)};
        const cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
        const cuuint32_t box[3] = {cuuint32_t(kv4_record(D)), 1u, cuuint32_t(kBlock)};
        if (!cache_map(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, sp.kv4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorUnknown;
    }
    auto go = [&](auto kern) {
        cudaError_t r = ensure_smem(kern, Geom::kTotal);
        if (r != cudaSuccess) return r;
        record_event(tm.begin, stream);
        r = launch_kernel(kern, dim3(unsigned(ctas)), dim3(Geom::kWarps * 32), Geom::kTotal, stream, true, 0, false, map, sp);
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
