// santa_shared.cu -- attention of a whole batch over a prefix that its sequences share.
//
// The queries of all sequences that read KV head h are R = batch * G rows against the same keys
// and values, so the prefix costs one read of K and V and two matrix products:
//   X = Q K^T / sqrt d,   E = 2^(X log2 e - M),   O = E V,   Z = E 1   (row by row),
// with a running maximum over blocks of keys.  Work is cut into units of (KV head, tile of rows,
// block of keys), and the units into equal contiguous stretches, one per CTA; a CTA writes the
// unnormalised (M, Z, O) of each item (KV head, tile) in its stretch, and a join kernel adds the
// parts of a row, with the row's own keys (window_kernel), in a fixed order.
//
// bf16 (shared_mma_kernel): both products on the tensor cores (tcgen05), 128 rows x 64 keys at a
// time.  K and V come by TMA through a ring of stages (boxes of 32 rows, so that a block may lie
// on two pages), S = Q K^T goes to tensor memory, a thread per row reads it, and E goes back to
// the tensor cores as the A operand of E V.  E is split into three bf16 parts by truncation (8 + 8 +
// 8 bits: exact), so a weight keeps its 24 bits; the parts are multiplied from the smallest on,
// each block into an accumulator that starts at zero and is added to O in registers by an fp32
// fma: a chain of thousands of additions on the tensor cores would lose bits to truncation.
// Two streams of four warps keep the tensor cores fed: while one stream's products run, the other
// forms weights.  They take two tiles of 128 rows over the same blocks or, with at most 128 rows,
// the even and the odd blocks of one tile.  A block's weights come in two halves of 32 keys, so that
// the products of the first run while the second is formed; a warp per stream issues its products.
//
// 64 sequences of 32 query and 8 KV heads of 128 over 32768 keys (34.4 GFLOP counted once, 68.7 with the
// parts of E; 134 MB): the whole call takes 85.5 us, of which this kernel has 57; per block of 64 keys
// and both tiles 3900 cycles, 2370 of them busy on the tensor cores.  It is bound by the chain of a
// block in each stream (S 1000 cycles after the last weights, first half 950, sums of the block before
// 850, second half 650, barriers): with two thirds of E V left out the call took no less, without the
// additions to O 3 us less.
//
// Tensor memory of a stream, 256 columns: O in 0 .. D - 1, S in 128 .. 191, the larger parts of E in
// 192 .. 223 and 224 .. 255; the smallest part has no room there and lies in shared memory.  So S of
// the next block can be formed as soon as E of this one is, before or beside E V.
//
// fp32 (shared_f32_kernel): 64 rows x 32 keys from shared memory on the FMA pipe.
#include "santa_split.cuh"
#include "santa_stream.cuh"
#include "santa_tcgen05.cuh"

namespace santa {

namespace {

constexpr int kRows = 128;     // rows of a stream's tile
constexpr int kKeys = 64;      // keys of a block
constexpr int kHalf = 32;      // keys of a TMA box
constexpr int kThreads = 384;  // streams 0 and 1 (four warps each); a producer, two warps of products, an idle one
// Registers per thread: launched with 168 (the file of 65536 over 384 threads), of which the last
// warpgroup gives back what the streams, with D sums and a block's values per thread, take.
constexpr int kLaunchRegs = 168, kStreamRegs = 224, kOtherRegs = 56;
static_assert(2 * kStreamRegs + kOtherRegs <= 3 * kLaunchRegs, "a larger share would wait forever");
template <int kRegs>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

template <int D>
struct MmaGeom {
    static constexpr int kBoxes = D / 64;                   // 128-byte columns of a row
    static constexpr int kTile = kKeys * D * 2;             // K or V of a block
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr size_t kQ = 0;                         // [2] tiles of Q
    static constexpr size_t kLow = size_t(2) * kRows * D * 2;      // [2] tiles of E's smallest part
    static constexpr size_t kStage0 = kLow + size_t(2) * kRows * kKeys * 2;
    static constexpr size_t kBars = kStage0 + size_t(kStages) * 2 * kTile;
    static constexpr size_t kTotal = kBars + (2 * kStages + 12) * 8 + kStages * 8 + 16;
    static_assert(kTotal <= 227 * 1024, "shared memory");
};

// The segments of a CTA's stretch: blocks blk .. blk + n - 1 of an item.  (Units are counted in
// 31 bits.)
struct Segments {
    int u, end;
    int item, blk, n, rows, first;  // rows of the item, from row `first` of the KV head on
    bool both;                      // the streams share the item's blocks
    __device__ __forceinline__ explicit Segments(const SharedParams &sp) {
        const int X = sp.p.Hkv * sp.tiles * sp.nb, q = X / sp.ctas, r = X - q * sp.ctas, c = blockIdx.x;
        u = q * c + min(c, r);  // as stretch_start
        end = u + q + (c < r ? 1 : 0);
        n = 0;
    }
    __device__ __forceinline__ bool next(const SharedParams &sp, int tile_rows, int streams) {
        u += n;
        if (u >= end) return false;
        item = u / sp.nb;
        blk = u - item * sp.nb;
        n = min(sp.nb - blk, end - u);
        first = item % sp.tiles * tile_rows * streams;
        rows = min(sp.rows - first, tile_rows * streams);
        both = streams == 2 && rows <= tile_rows;
        return true;
    }
    // blocks of stream t, and the place of its i-th among the segment's
    __device__ __forceinline__ int count(int t) const { return both ? (n + 1 - t) / 2 : n; }
    __device__ __forceinline__ int place(int t, int i) const { return both ? 2 * i + t : i; }
};

// Logits of keys that do not count become -inf (their weight 0), whatever they hold.
__device__ __forceinline__ void drop(float (&x)[16], uint32_t seen) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
        if (!(seen >> j & 1)) x[j] = -INFINITY;
}
// A row's weights of 32 keys (x, y: their raw logits), as the parts of E: two in tensor memory from
// columns hi_at and mid_at on, the smallest at `low` (the row's 128 bytes in the swizzle of the operand),
// pieces of 16 bytes from `piece` on.  Adds them to sum.
__device__ __forceinline__ void half_weights(float (&x)[16], float (&y)[16], float scale2, float ref, uint32_t hi_at,
                                             uint32_t mid_at, unsigned char *low, int piece, int r, float2 &sum) {
    const float2 scale = make_float2(scale2, scale2), shift = make_float2(-ref, -ref);
#pragma unroll
    for (int d = 0; d < 2; ++d) {
        uint32_t hi[8], mid[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float2 e = __ffma2_rn(d ? make_float2(y[2 * j], y[2 * j + 1]) : make_float2(x[2 * j], x[2 * j + 1]), scale, shift);
            e = make_float2(ex2(e.x), ex2(e.y));
            sum = __fadd2_rn(sum, e);
            // what a part leaves over is exact
            uint32_t u = __float_as_uint(e.x), v = __float_as_uint(e.y);
            hi[j] = __byte_perm(u, v, 0x7632);
            e = __fadd2_rn(e, make_float2(-__uint_as_float(u & 0xffff0000u), -__uint_as_float(v & 0xffff0000u)));
            u = __float_as_uint(e.x), v = __float_as_uint(e.y);
            mid[j] = __byte_perm(u, v, 0x7632);
            e = __fadd2_rn(e, make_float2(-__uint_as_float(u & 0xffff0000u), -__uint_as_float(v & 0xffff0000u)));
            lo[j] = __byte_perm(__float_as_uint(e.x), __float_as_uint(e.y), 0x7632);
        }
        tmem_store8(hi_at + 8 * d, hi);
        tmem_store8(mid_at + 8 * d, mid);
        *reinterpret_cast<uint4 *>(low + (((piece + 2 * d) ^ (r & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(low + (((piece + 2 * d + 1) ^ (r & 7)) << 4)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
}
// O = O * sc + the block's sums.
template <int D>
__device__ __forceinline__ void add_sums(uint32_t base, float2 (&O)[D / 2], float sc) {
    const float2 sc2 = make_float2(sc, sc);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
        float x[16], y[16];
        tmem_load16(base + 32 * c, x);
        tmem_load16(base + 32 * c + 16, y);
        tmem_wait(x, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            O[16 * c + j] = __ffma2_rn(O[16 * c + j], sc2, make_float2(x[2 * j], x[2 * j + 1]));
            O[16 * c + 8 + j] = __ffma2_rn(O[16 * c + 8 + j], sc2, make_float2(y[2 * j], y[2 * j + 1]));
        }
    }
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    shared_mma_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ SharedParams sp) {
    using Geo = MmaGeom<D>;
    constexpr int NS = Geo::kStages;
    const Params &p = sp.p;
    const int warp = __shfl_sync(kFull, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // uniform
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + Geo::kBars), *empty = full + NS;
    // per stream: S is there; E is there, half by half; O is there; Q is there; all products have ended
    uint64_t *sready = empty + NS, *eready = sready + 2, *oready = eready + 4, *qready = oready + 2, *fin = qready + 2;
    uint2 *valid = reinterpret_cast<uint2 *>(fin + 2);  // a stage's keys that count, a bit each
    uint32_t *tmem_at = reinterpret_cast<uint32_t *>(valid + NS);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);  // either stream's products, or one's and an arrive for the other
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sready[t], 1);
            mbar_init(&eready[2 * t], kRows);
            mbar_init(&eready[2 * t + 1], kRows);
            mbar_init(&oready[t], 1);
            mbar_init(&qready[t], kRows);
            mbar_init(&fin[t], 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    if (warp == 9) tmem_alloc(tmem_at);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = __shfl_sync(kFull, *tmem_at, 0);
    pdl_wait();
    pdl_launch_dependents();

    auto give_up = [&]() { raise_flag(p, SANTA_ERR_TIMEOUT | (5u << 8)); };  // location code 5
    Segments sg(sp);
    int it = 0;  // blocks of the CTA before this segment

    if (warp >= 8) fewer_registers<kOtherRegs>();
    if (warp == 11) {
    } else if (warp == 8) {  // producer
        bool ok = true;
        while (ok && sg.next(sp, kRows, 2)) {
            const int kvh = sg.item / sp.tiles;
            int row = -1, count = 0;  // lane l: half l of the next 16 blocks, its first row and its keys
            for (int j = 0; ok && j < sg.n; ++j, ++it) {
                if (j % 16 == 0) {
                    const long long key = ((long long)(sg.blk + j) * 2 + lane) * kHalf;
                    row = -1;
                    count = 0;
                    if (key < sp.len && lane < 2 * (sg.n - j)) {
                        const long long r = kPaged ? key_row<kPaged>(p, 0, 0, int(key)) : sp.start + key;
                        row = int(r);
                        count = r < 0 ? 0 : int(min((long long)kHalf, sp.len - key));
                    }
                }
                const int s = it % NS, l = j % 16 * 2;
                const int r0 = __shfl_sync(kFull, row, l), r1 = __shfl_sync(kFull, row, l + 1);
                const int n0 = __shfl_sync(kFull, count, l), n1 = __shfl_sync(kFull, count, l + 1);
                if (lane == 0) {
                    ok = mbar_wait(&empty[s], ((it / NS) & 1) ^ 1);
                    if (ok) {
                        valid[s] = make_uint2(n0 >= 32 ? kFull : (1u << n0) - 1, n1 >= 32 ? kFull : (1u << n1) - 1);
                        const uint32_t bytes = ((n0 > 0) + (n1 > 0)) * kHalf * D * 2 * 2;
                        if (bytes)
                            mbar_arrive_expect_tx(&full[s], bytes);
                        else
                            mbar_arrive(&full[s]);
                        unsigned char *k = smem + Geo::kStage0 + size_t(s) * 2 * Geo::kTile, *v = k + Geo::kTile;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if ((half ? n1 : n0) == 0) continue;
                            const int r = half ? r1 : r0;
#pragma unroll
                            for (int bx = 0; bx < Geo::kBoxes; ++bx)
                                tma_load_3d(k + bx * kKeys * 128 + half * kHalf * 128, &kmap, &full[s], bx * 64, kvh, r);
#pragma unroll
                            for (int bx = 0; bx < Geo::kBoxes; ++bx)
                                tma_load_3d(v + bx * kKeys * 128 + half * kHalf * 128, &vmap, &full[s], bx * 64, kvh, r);
                        }
                    } else {
                        give_up();
                    }
                }
                ok = __shfl_sync(kFull, ok, 0);
            }
        }
        if (lane == 0) {  // the copies in flight land before the CTA ends, whatever the others did
            const long long t0 = clock64();
            for (int i = it > NS ? it - NS : 0; i < (ok ? it : it - 1); ++i)
                while (!mbar_try_wait(&full[i % NS], (i / NS) & 1) && clock64() - t0 < kWaitCycles) {
                }
        }
    } else if (warp >= 9) {  // products of stream t: the warp as one, an elected lane issues
        const int t = warp - 9;
        bool ok = true;
        uint32_t phQ = 0, ph = 0;
        constexpr uint32_t kind_s = mma_kind(kRows, kKeys, false), kind_o = mma_kind(kRows, D, true);
        const uint32_t base = tmem + t * 256;
        const uint64_t q = operand(smem_addr(smem + Geo::kQ) + t * kRows * D * 2, 16, 1024);
        const uint64_t k0 = operand(smem_addr(smem + Geo::kStage0), 16, 1024);
        const uint64_t v0 = operand(smem_addr(smem + Geo::kStage0) + Geo::kTile, kKeys * 128, 1024);
        const uint64_t low = operand(smem_addr(smem + Geo::kLow) + t * kRows * kKeys * 2, 16, 1024);
        auto wait = [&](uint64_t *bar, uint32_t phase) { return bool(__all_sync(kFull, mbar_wait(bar, phase))); };
        // S of the stream's i-th block, whose K is there
        auto scores = [&](int i) {
            const int s = (it + sg.place(t, i)) % NS;
            const uint64_t k = k0 + __shfl_sync(kFull, s * (2 * Geo::kTile / 16), 0);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(base + 128, q + ((ks >> 2) * kRows * 128 + (ks & 3) * 32) / 16,
                           k + ((ks >> 2) * kKeys * 128 + (ks & 3) * 32) / 16, kind_s, ks > 0);
                mma_commit(&sready[t]);
            }
            __syncwarp();
        };
        auto arrived = [&](int i, bool now) {  // K and V of the i-th block; `now`: without waiting
            const int block = it + sg.place(t, i);
            const bool there = now ? bool(__all_sync(kFull, mbar_try_wait(&full[block % NS], (block / NS) & 1)))
                                   : wait(&full[block % NS], (block / NS) & 1);
            tc_after_sync();
            return there;
        };
        // O of half h of the i-th block
        auto sums = [&](int i, int h) {
            const int s = (it + sg.place(t, i)) % NS;
            const uint64_t v = v0 + __shfl_sync(kFull, s * (2 * Geo::kTile / 16), 0);
            if (elect_one()) {
#pragma unroll
                for (int part = 0; part < 3; ++part)  // the smallest first
#pragma unroll
                    for (int k2 = 0; k2 < kHalf / 16; ++k2) {
                        const int ks = h * (kHalf / 16) + k2;
                        if (part == 0)
                            mma_ss(base, low + ks * 32 / 16, v + ks * 16 * 128 / 16, kind_o, h + k2 > 0);
                        else
                            mma_ts(base, base + (part == 1 ? 224 : 192) + ks * 8, v + ks * 16 * 128 / 16, kind_o, true);
                    }
                if (h == 1) {
                    mma_commit(&oready[t]);
                    mma_commit(&empty[s]);
                    if (sg.both) mbar_arrive(&empty[s]);
                }
            }
            __syncwarp();
        };
        while (ok && sg.next(sp, kRows, 2)) {
            const int n = sg.count(t);
            if (n > 0) {
                ok = wait(&qready[t], phQ) && arrived(0, false);
                phQ ^= 1;
                if (ok) scores(0);
            }
#pragma unroll 1
            for (int i = 0; ok && i < n; ++i) {
                ok = wait(&eready[2 * t], ph);
                if (!ok) break;
                tc_after_sync();
                sums(i, 0);
                ok = wait(&eready[2 * t + 1], ph);
                ph ^= 1;
                if (!ok) break;
                tc_after_sync();
                // the next S first, unless its K is late
                const bool next = i + 1 < n, early = next && arrived(i + 1, true);
                if (early) scores(i + 1);
                sums(i, 1);
                if (next && !early) {
                    ok = arrived(i + 1, false);
                    if (ok) scores(i + 1);
                }
            }
            it += sg.n;
        }
        if (!ok && lane == 0) give_up();
        __syncwarp();
        if (elect_one()) mma_commit(&fin[t]);  // every product has ended before tensor memory is given back
        __syncwarp();
        if (!wait(&fin[t], 0) && lane == 0) give_up();
        __syncwarp();
    } else {  // weights
        more_registers<kStreamRegs>();
        const int t = warp >> 2, r = threadIdx.x & (kRows - 1);
        const uint32_t base = tmem + t * 256 + (uint32_t(warp & 3) << 21);
        const float scale2 = p.scale * 1.4426950408889634f;  // logits in base 2
        bool ok = true;
        uint32_t ph = 0;
        while (ok && sg.next(sp, kRows, 2)) {
            const int kvh = sg.item / sp.tiles, row0 = sg.first + (sg.both ? 0 : t * kRows);
            const int rows = sg.both ? sg.rows : min(kRows, sg.rows - t * kRows);  // may be <= 0
            const int n = sg.count(t);
            // the stream's tile of Q, rows of zeros behind the last: a piece of 16 bytes per thread and round
            if (n > 0) {
                constexpr int kVecs = D / 8, kRounds = kRows * kVecs / kRows;
                const int vec = r % kVecs;
                uint4 x[kRounds];
#pragma unroll
                for (int u = 0; u < kRounds; ++u) {
                    const int qr = r / kVecs + u * (kRows / kVecs);
                    const int b = (row0 + qr) / p.G, g = (row0 + qr) - b * p.G;
                    x[u] = qr < rows ? load(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) +
                                                                            (size_t(b) * p.Hq + kvh * p.G + g) * D) + vec)
                                     : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < kRounds; ++u) {
                    const int qr = r / kVecs + u * (kRows / kVecs);
                    *reinterpret_cast<uint4 *>(smem + Geo::kQ + size_t(t) * kRows * D * 2 + (vec >> 3) * kRows * 128 +
                                               qr * 128 + (((vec & 7) ^ (qr & 7)) << 4)) = x[u];
                }
            }
            if (n > 0) {  // (a stream that has no block must not run ahead of its barrier's phase)
                fence_proxy_async_smem();
                tc_before_sync();
                mbar_arrive(&qready[t]);
            }

            float2 O[D / 2];
            float M = -INFINITY, Z = 0.f;
#pragma unroll
            for (int i = 0; i < D / 2; ++i) O[i] = make_float2(0.f, 0.f);
            float sc = 0.f;  // of the block before
            for (int i = 0; i < n; ++i) {
                const int b = it + sg.place(t, i), s = b % NS;
                // the stage stays until this block's sums are formed, so its barrier's phase does too
                ok = mbar_wait(&full[s], (b / NS) & 1);
                if (!ok) break;
                const uint2 seen2 = valid[s];
                ok = mbar_wait(&sready[t], ph);
                if (!ok) break;
                tc_after_sync();
                const bool whole = (seen2.x & seen2.y) == kFull;
                unsigned char *low = smem + Geo::kLow + size_t(t * kRows + r) * kKeys * 2;
                float2 sum = make_float2(0.f, 0.f);
                float ref, sc_next;
                {
                    float x[16], y[16];  // the first half
                    {
                        float u[16], v[16];
                        tmem_load16(base + 160, u);
                        tmem_load16(base + 176, v);
                        tmem_load16(base + 128, x);
                        tmem_load16(base + 144, y);
                        tmem_wait(u, v);
                        tmem_arrived(x, y);
                        if (!whole) {
                            drop(x, seen2.x);
                            drop(y, seen2.x >> 16);
                            drop(u, seen2.y);
                            drop(v, seen2.y >> 16);
                        }
                        float m = M;
#pragma unroll
                        for (int j = 0; j < 16; ++j) m = fmaxf(fmaxf(m, fmaxf(x[j], y[j])), fmaxf(u[j], v[j]));
                        ref = m == -INFINITY ? 0.f : m * scale2;
                        sc_next = ex2(fmaf(M, scale2, -ref));
                        M = m;
                    }
                    // (E of the block before has been read where S of this one is there: its products came first)
                    half_weights(x, y, scale2, ref, base + 192, base + 224, low, 0, r, sum);
                }
                if (i > 0) {
                    ok = mbar_wait(&oready[t], ph ^ 1);
                    if (!ok) break;
                    tc_after_sync();
                    add_sums<D>(base, O, sc);
                }
                sc = sc_next;
                if (!whole) {  // weight 0 times a row that holds anything
                    unsigned char *v = smem + Geo::kStage0 + size_t(s) * 2 * Geo::kTile + Geo::kTile;
                    for (int j = r; j < kKeys * Geo::kBoxes * 8; j += kRows) {
                        const int key = (j >> 3) % kKeys, bx = (j >> 3) / kKeys;
                        if (!((key < 32 ? seen2.x : seen2.y) >> (key & 31) & 1))
                            *reinterpret_cast<uint4 *>(v + bx * kKeys * 128 + key * 128 + (j & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                tmem_wait_store();
                tc_before_sync();
                mbar_arrive(&eready[2 * t]);
                {
                    float x[16], y[16];
                    tmem_load16(base + 160, x);
                    tmem_load16(base + 176, y);
                    tmem_wait(x, y);
                    if (!whole) {
                        drop(x, seen2.y);
                        drop(y, seen2.y >> 16);
                    }
                    half_weights(x, y, scale2, ref, base + 208, base + 240, low, 4, r, sum);
                }
                Z = fmaf(Z, sc, sum.x + sum.y);
                fence_proxy_async_smem();
                tmem_wait_store();
                tc_before_sync();
                mbar_arrive(&eready[2 * t + 1]);
                ph ^= 1;
            }
            if (ok && n > 0) {
                ok = mbar_wait(&oready[t], ph ^ 1);
                tc_after_sync();
                if (ok) add_sums<D>(base, O, sc);
            }
            if (!ok) break;
            if (r < rows) {
                const size_t at = (size_t(sg.item + blockIdx.x) * 2 + t) * kRows + r;
                sp.mz[at] = make_float2(M == -INFINITY ? M : M * scale2, Z);
                if (n > 0)  // whole sectors of 32 bytes per thread
#pragma unroll
                    for (int i = 0; i < D / 8; ++i)
                        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(sp.o + at * D + 8 * i),
                                     "f"(O[4 * i].x), "f"(O[4 * i].y), "f"(O[4 * i + 1].x), "f"(O[4 * i + 1].y),
                                     "f"(O[4 * i + 2].x), "f"(O[4 * i + 2].y), "f"(O[4 * i + 3].x), "f"(O[4 * i + 3].y)
                                     : "memory");
            }
            it += sg.n;
        }
        if (!ok) give_up();
        tc_before_sync();
    }
    __syncthreads();
    tc_after_sync();
    if (warp == 9) tmem_free(tmem);
}

// ---------------------------------------------------------------- fp32

constexpr int kF32Rows = 64, kF32Keys = 32, kF32Threads = 256;

template <int D>
struct F32Geom {
    static constexpr int kStride = D + 4;  // rows start 16 bytes apart from a multiple of 128
    static constexpr size_t kK = size_t(kF32Rows) * kStride * 4, kV = kK + size_t(kF32Keys) * kStride * 4;
    static constexpr size_t kE = kV + size_t(kF32Keys) * kStride * 4, kEStride = kF32Keys + 1;
    static constexpr size_t kTotal = kE + size_t(kF32Rows) * kEStride * 4;
};

// Thread (ty, tx) of 16 x 16: rows 4 ty .. + 3 of the tile, keys tx and tx + 16 of the block, then
// the elements 4 tx + 64 i .. + 3 of the sums.  The next block is loaded while this one is used.
template <int D, bool kPaged>
__global__ void __launch_bounds__(kF32Threads, 1) shared_f32_kernel(const __grid_constant__ SharedParams sp) {
    using Geo = F32Geom<D>;
    constexpr int S = Geo::kStride, kE = D / 64, kPer = kF32Keys * D / 4 / kF32Threads;
    const Params &p = sp.p;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    extern __shared__ __align__(1024) unsigned char smem[];
    float *Q = reinterpret_cast<float *>(smem), *K = reinterpret_cast<float *>(smem + Geo::kK);
    float *V = reinterpret_cast<float *>(smem + Geo::kV), *E = reinterpret_cast<float *>(smem + Geo::kE);
    const float scale2 = p.scale * 1.4426950408889634f;
    pdl_wait();
    pdl_launch_dependents();
    Segments sg(sp);
    while (sg.next(sp, kF32Rows, 1)) {
        const int kvh = sg.item / sp.tiles;
        __syncthreads();  // the last segment's reads of Q
        for (int i = threadIdx.x; i < kF32Rows * D / 4; i += kF32Threads) {
            const int r = i / (D / 4), c = i % (D / 4);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < sg.rows) {
                const int b = (sg.first + r) / p.G, g = (sg.first + r) - b * p.G;
                x = load(reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) +
                                                          (size_t(b) * p.Hq + kvh * p.G + g) * D) + c);
            }
            *reinterpret_cast<float4 *>(Q + r * S + 4 * c) = x;
        }
        float4 nk[kPer], nv[kPer];
        unsigned next = 0;  // keys of the loaded block that count: bit per this thread's pieces
        auto fetch = [&](int blk) {
            next = 0;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = threadIdx.x + u * kF32Threads, key = blk * kF32Keys + i / (D / 4), c = i % (D / 4);
                const long long row = key < sp.len ? kPaged ? key_row<kPaged>(p, 0, 0, key) : sp.start + key : -1;
                nk[u] = nv[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0) {
                    const size_t at = (size_t(row) * p.Hkv + kvh) * D;
                    nk[u] = load(reinterpret_cast<const float4 *>(static_cast<const float *>(p.k) + at) + c);
                    nv[u] = load(reinterpret_cast<const float4 *>(static_cast<const float *>(p.v) + at) + c);
                    next |= 1u << u;
                }
            }
        };
        float4 O[4][kE];
        float M[4], Z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            M[i] = -INFINITY;
            Z[i] = 0.f;
#pragma unroll
            for (int j = 0; j < kE; ++j) O[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __shared__ unsigned seen[kF32Keys];
        fetch(sg.blk);
        for (int j = 0; j < sg.n; ++j) {
            __syncthreads();  // K, V and E of the block before are done with
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const int i = threadIdx.x + u * kF32Threads, key = i / (D / 4), c = i % (D / 4);
                *reinterpret_cast<float4 *>(K + key * S + 4 * c) = nk[u];
                *reinterpret_cast<float4 *>(V + key * S + 4 * c) = nv[u];
                if (c == 0) seen[key] = next >> u & 1;
            }
            __syncthreads();
            if (j + 1 < sg.n) fetch(sg.blk + j + 1);
            float2 a[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i][0] = a[i][1] = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < D / 4; ++c) {
                const float4 k0 = *reinterpret_cast<const float4 *>(K + tx * S + 4 * c);
                const float4 k1 = *reinterpret_cast<const float4 *>(K + (tx + 16) * S + 4 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 q = *reinterpret_cast<const float4 *>(Q + (4 * ty + i) * S + 4 * c);
                    a[i][0] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k0.x, k0.y), a[i][0]);
                    a[i][0] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k0.z, k0.w), a[i][0]);
                    a[i][1] = __ffma2_rn(make_float2(q.x, q.y), make_float2(k1.x, k1.y), a[i][1]);
                    a[i][1] = __ffma2_rn(make_float2(q.z, q.w), make_float2(k1.z, k1.w), a[i][1]);
                }
            }
            const bool in0 = seen[tx], in1 = seen[tx + 16];
            float sc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = in0 ? (a[i][0].x + a[i][0].y) * scale2 : -INFINITY;
                const float x1 = in1 ? (a[i][1].x + a[i][1].y) * scale2 : -INFINITY;
                float m = fmaxf(x0, x1);
#pragma unroll
                for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
                m = fmaxf(m, M[i]);
                const float ref = m == -INFINITY ? 0.f : m;
                sc[i] = ex2(M[i] - ref);
                M[i] = m;
                const float e0 = ex2(x0 - ref), e1 = ex2(x1 - ref);
                Z[i] = fmaf(Z[i], sc[i], e0 + e1);  // of this thread's keys
                E[(4 * ty + i) * Geo::kEStride + tx] = e0;
                E[(4 * ty + i) * Geo::kEStride + tx + 16] = e1;
            }
            __syncwarp();  // a row's weights are one warp's
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < kE; ++u)
                    O[i][u] = make_float4(O[i][u].x * sc[i], O[i][u].y * sc[i], O[i][u].z * sc[i], O[i][u].w * sc[i]);
#pragma unroll 4
            for (int key = 0; key < kF32Keys; ++key) {
                float4 v[kE];
#pragma unroll
                for (int u = 0; u < kE; ++u) v[u] = *reinterpret_cast<const float4 *>(V + key * S + 4 * tx + 64 * u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = E[(4 * ty + i) * Geo::kEStride + key];
#pragma unroll
                    for (int u = 0; u < kE; ++u)
                        O[i][u] = make_float4(fmaf(e, v[u].x, O[i][u].x), fmaf(e, v[u].y, O[i][u].y),
                                              fmaf(e, v[u].z, O[i][u].z), fmaf(e, v[u].w, O[i][u].w));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) Z[i] += __shfl_xor_sync(kFull, Z[i], o);
            const int r = 4 * ty + i;
            if (r >= sg.rows) continue;
            const size_t at = size_t(sg.item + blockIdx.x) * kF32Rows + r;
            if (tx == 0) sp.mz[at] = make_float2(M[i], Z[i]);
#pragma unroll
            for (int u = 0; u < kE; ++u) reinterpret_cast<float4 *>(sp.o + at * D + 64 * u)[tx] = O[i][u];
        }
    }
}

// ---------------------------------------------------------------- join

constexpr int kJoinThreads = 128;
constexpr int kJoinParts = 2 * kSplitCtaBound;

// One row: the parts of its item, and its own keys' state.  (x, y) = (query head, sequence).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) shared_join_kernel(const __grid_constant__ SharedParams sp, int tile_rows,
                                                                   int streams) {
    constexpr int kCols = D / 4, kGroups = kJoinThreads / kCols, kPer = (kJoinParts + kJoinThreads - 1) / kJoinThreads;
    const Params &p = sp.p;
    const int hq = blockIdx.x, b = blockIdx.y, kvh = hq / p.G, r = b * p.G + hq - kvh * p.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float coef[kJoinParts], red[2][kJoinThreads / 32];
    __shared__ float4 sums[kGroups][kCols];
    const int full = tile_rows * streams, tile = r / full, within = r - tile * full;
    const bool both = streams == 2 && min(sp.rows - tile * full, full) <= tile_rows;
    const int stream = both ? 0 : within / tile_rows, row = within - stream * tile_rows;
    const long long X = (long long)p.Hkv * sp.tiles * sp.nb;
    const int item = kvh * sp.tiles + tile;
    const int c0 = stretch_of(X, sp.ctas, (long long)item * sp.nb);
    const int c1 = stretch_of(X, sp.ctas, (long long)(item + 1) * sp.nb - 1);
    const int parts = (c1 - c0 + 1) << int(both);
    auto index = [&](int j) {
        const int cta = c0 + (j >> int(both)), t = both ? j & 1 : stream;
        return (size_t(item + cta) * streams + t) * tile_rows + row;
    };
    pdl_wait();
    pdl_launch_dependents();
    const size_t at = size_t(b) * p.Hq + hq;
    const float2 own = sp.own_mz ? load(sp.own_mz + at) : make_float2(-INFINITY, 0.f);
    float2 mz[kPer];
    float M = own.x;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int j = threadIdx.x + u * kJoinThreads;
        mz[u] = j < parts ? load(sp.mz + index(j)) : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, mz[u].x);
    }
    M = warp_max(M);
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
    for (int i = 0; i < kJoinThreads / 32; ++i) M = fmaxf(M, red[0][i]);
    const float ref = M == -INFINITY ? 0.f : M;
    float Z = 0.f;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
        const int j = threadIdx.x + u * kJoinThreads;
        const float c = ex2(mz[u].x - ref);
        Z = fmaf(mz[u].y, c, Z);
        if (j < parts) coef[j] = c;
    }
    Z = warp_sum(Z);
    if (lane == 0) red[1][warp] = Z;
    __syncthreads();
    const float own_z = own.y * ex2(own.x - ref);
    Z = own_z;
    for (int i = 0; i < kJoinThreads / 32; ++i) Z += red[1][i];
    const int col = threadIdx.x % kCols, grp = threadIdx.x / kCols;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = grp; j < parts; j += kGroups) {
        const float c = coef[j];
        if (c == 0.f) continue;  // a part without mass may hold no sums
        const float4 x = load(reinterpret_cast<const float4 *>(sp.o + index(j) * D) + col);
        acc.x = fmaf(c, x.x, acc.x);
        acc.y = fmaf(c, x.y, acc.y);
        acc.z = fmaf(c, x.z, acc.z);
        acc.w = fmaf(c, x.w, acc.w);
    }
    sums[grp][col] = acc;
    __syncthreads();
    if (threadIdx.x < kCols) {
        float4 *out = reinterpret_cast<float4 *>(p.out + at * D) + col;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (own_z != 0.f) {
            const float4 x = *out;
            acc = make_float4(x.x * own_z, x.y * own_z, x.z * own_z, x.w * own_z);
        }
        for (int g = 0; g < kGroups; ++g) {
            const float4 x = sums[g][col];
            acc.x += x.x;
            acc.y += x.y;
            acc.z += x.z;
            acc.w += x.w;
        }
        const float inv = Z == 0.f ? 0.f : 1.f / Z;
        *out = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    }
}

template <int D, bool kPaged>
cudaError_t launch_mma(const SharedParams &sp, cudaStream_t stream) {
    const Params &p = sp.p;
    CUtensorMap maps[2];
    for (int i = 0; i < 2; ++i) {  // [rows][Hkv][d]: boxes of 128 bytes of one head's row x 32 rows
        const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(p.Hkv), cuuint64_t(p.total_tokens)};
        const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(p.Hkv) * D * 2};
        const cuuint32_t box[3] = {64u, 1u, cuuint32_t(kHalf)};
        if (!cache_map(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, i ? p.v : p.k, dims, strides, box,
                       CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorUnknown;
    }
    auto kern = shared_mma_kernel<D, kPaged>;
    cudaError_t r = ensure_smem(kern, MmaGeom<D>::kTotal);
    static bool checked = false;  // the streams' registers come out of those the kernel is launched with
    if (r == cudaSuccess && !checked) {
        cudaFuncAttributes a;
        r = cudaFuncGetAttributes(&a, kern);
        if (r == cudaSuccess && a.numRegs < kLaunchRegs) r = cudaErrorNotSupported;
        checked = r == cudaSuccess;
    }
    if (r != cudaSuccess) return r;
    return launch_kernel(kern, dim3(unsigned(sp.ctas)), dim3(kThreads), MmaGeom<D>::kTotal, stream, true, 0, false, maps[0],
                         maps[1], sp);
}

template <int D>
cudaError_t launch_f32(const SharedParams &sp, cudaStream_t stream) {
    auto go = [&](auto kern) {
        const cudaError_t r = ensure_smem(kern, F32Geom<D>::kTotal);
        if (r != cudaSuccess) return r;
        return launch_kernel(kern, dim3(unsigned(sp.ctas)), dim3(kF32Threads), F32Geom<D>::kTotal, stream, true, 0, false,
                             sp);
    };
    return sp.p.page_table ? go(shared_f32_kernel<D, true>) : go(shared_f32_kernel<D, false>);
}

// Blocks of keys per CTA, at least.  bf16: one leaves no SM to the own keys' kernel, which runs beside
// (4 sequences, 1000 keys: 16.4 us with 1, 12.3 with 2, 13.2 with 4); fp32 blocks are smaller and take
// longer (8 sequences, 1023 keys of 64: 11.6 us with 1, 12.9 with 2, 17.8 with 4).
constexpr int min_blocks(int dtype) { return dtype == SANTA_BF16 ? 2 : 1; }

}  // namespace

cudaError_t launch_shared(SharedParams &sp, int dtype, cudaStream_t stream, const Timing &tm) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long X = (long long)sp.p.Hkv * sp.tiles * sp.nb, least = min_blocks(dtype), most = (X + least - 1) / least;
    if (X > 0x7fffffffLL) return cudaErrorNotSupported;
    const int ctas = sms < kSplitCtaBound ? sms : kSplitCtaBound;
    sp.ctas = most < ctas ? int(most) : ctas;
    record_event(tm.begin, stream);
    if (dtype == SANTA_BF16 && sp.p.page_table)
        e = sp.p.D == 128 ? launch_mma<128, true>(sp, stream) : launch_mma<64, true>(sp, stream);
    else if (dtype == SANTA_BF16)
        e = sp.p.D == 128 ? launch_mma<128, false>(sp, stream) : launch_mma<64, false>(sp, stream);
    else
        e = sp.p.D == 128 ? launch_f32<128>(sp, stream) : launch_f32<64>(sp, stream);
    record_event(tm.end, stream);
    return e;
}

cudaError_t launch_shared_join(const SharedParams &sp, int dtype, cudaStream_t stream) {
    const dim3 grid(unsigned(sp.p.Hq), unsigned(sp.p.B));
    auto go = [&](auto kern) {
        return launch_kernel(kern, grid, dim3(kJoinThreads), 0, stream, true, 0, false, sp, shared_rows(dtype),
                             shared_streams(dtype));
    };
    return sp.p.D == 128 ? go(shared_join_kernel<128>) : go(shared_join_kernel<64>);
}

}  // namespace santa
