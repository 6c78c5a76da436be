// santa_kv4_store.cu -- the 4-bit cache's append and read.
//
// A row (K or V of one token and KV head) is held by D / 16 lanes, two blocks of 8 elements
// each, l and l + D / 16; the blocks alternate between the row's D / 64 groups, so a lane's
// two are of one group, and the lanes of a group are those with one value of l mod (D / 64).
// Append: minimum and maximum over the group (two shuffles each), minimum and scale rounded
// to fp16 first, so that the codes are formed against the values that a reader will use:
//   code = rn((x - min) / scale) held to 0 .. 15.
// 8 codes are one 32-bit word of the record.  What is stored is defined by single
// IEEE operations in fp32 (no fused multiply-add, division rounded to nearest), so the codes
// do not depend on how the kernel is compiled.  The division itself is only done where it
// matters: with r an approximate reciprocal (2^-23) over 15, 15 (x - min) r is off from the
// rounded quotient by less than 6 2^-24 of itself, 5.6e-6 for quotients below 15.5, so a result
// further than 1e-5 from the middle between two codes rounds as the quotient does.
//
// A prompt of 8191 tokens, 8 heads of 128, is 43 MB in and out for either direction (6.3 us at
// the copy rate): 15.0 us and 9.4 us (2.9 and 4.6 TB/s), at first 22 each.  Neither is bound by one
// thing: the warps' 9.8 and 5.0 million instructions are 7.8 and 4.0 us of every scheduler's time at
// the top clock, 0.59 and 0.58 of the cycles issue one, and half (append) or more (read) of a
// warp's time between two of them is the wait for its loads.  What brought them down: two blocks per lane instead
// of one (20 -> 15 and 12 -> 9.5), packed minimum and maximum, no IEEE division, rounding and packing
// by the low bits of a large float, and codes read as fp16 subnormals.  Two or four rows in flight
// per lane were tried and brought no gain.
#include <cuda_fp16.h>

#include "santa_rows.cuh"
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kStoreThreads = 256;
constexpr float kHalfMax = 65504.f;

// The rows of a token are K of its KV heads, then V; D / 16 lanes take one.
struct RowOf {
    int t, h, which;
    bool live;
};
__device__ __forceinline__ RowOf row_of(const StoreParams &p, int lanes) {
    const long long row = ((long long)blockIdx.x * kStoreThreads + threadIdx.x) / lanes;
    const int per = 2 * p.Hkv;
    RowOf r;
    const long long t = row >> 31 ? row / per : (long long)(unsigned(row) / unsigned(per));
    r.live = t < p.tokens;
    r.t = r.live ? int(t) : 0;
    const int i = r.live ? int(row - t * per) : 0;
    r.which = i >= p.Hkv;
    r.h = i - r.which * p.Hkv;
    return r;
}

// The token's slot, -1 if it has none (padding, behind the last token, or beyond the cache: flagged).
__device__ __forceinline__ long long slot_of(const StoreParams &p, const RowOf &r) {
    if (!r.live) return -1;
    const long long slot = p.slot_map ? load(p.slot_map + r.t) : r.t;
    if (slot >= p.total_tokens) {
        if (p.err) atomicOr(p.err, SANTA_ERR_SLOT);
        return -1;
    }
    return slot;
}

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// (minimum, -maximum) of a lane's two blocks and then of the group's lanes (those whose index
// differs in bits >= log2 kGroups); NaN if there is one.
template <int kGroups, int kL>
__device__ __forceinline__ float2 extremes(const uint4 (&raw)[2][1], const float (&)[2][8], uint16_t) {
    const uint32_t w[8] = {raw[0][0].x, raw[0][0].y, raw[0][0].z, raw[0][0].w,
                           raw[1][0].x, raw[1][0].y, raw[1][0].z, raw[1][0].w};
    __nv_bfloat162 lo = *reinterpret_cast<const __nv_bfloat162 *>(&w[0]), hi = lo;
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        lo = __hmin2_nan(lo, *reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
        hi = __hmax2_nan(hi, *reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
    }
    // (lo, -hi) in one register: exact, because extremes of bf16 values are bf16
    __nv_bfloat162 m = __halves2bfloat162(__hmin_nan(__low2bfloat16(lo), __high2bfloat16(lo)),
                                          __hneg(__hmax_nan(__low2bfloat16(hi), __high2bfloat16(hi))));
#pragma unroll
    for (int o = kGroups; o < kL; o <<= 1) m = __hmin2_nan(m, __shfl_xor_sync(kFull, m, o));
    return __bfloat1622float2(m);
}
template <int kGroups, int kL>
__device__ __forceinline__ float2 extremes(const uint4 (&)[2][2], const float (&x)[2][8], float) {
    float lo = x[0][0], hi = -x[0][0];
#pragma unroll
    for (int j = 1; j < 16; ++j) {
        lo = min_nan(lo, x[j / 8][j % 8]);
        hi = min_nan(hi, -x[j / 8][j % 8]);
    }
#pragma unroll
    for (int o = kGroups; o < kL; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
        hi = min_nan(hi, __shfl_xor_sync(kFull, hi, o));
    }
    return make_float2(lo, hi);
}

// The codes of a block, element j at bits 4 j.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float base, float scale) {
    constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer in the low bits
    if (!(scale > 0.f)) return 0u;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    inv *= 1.0f / 15.0f;
    float n[8], off = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 d = __fadd2_rn(make_float2(x[j], x[j + 1]), make_float2(-base, -base));
        // the quotient's fifteenth held to 0 .. 1 (the minimum's rounding can leave d < 0)
        const float2 q = make_float2(__saturatef(d.x * inv), __saturatef(d.y * inv));
        const float2 r = __ffma2_rn(q, make_float2(15.f, 15.f), make_float2(kMagic, kMagic));
        const float2 e = __fadd2_rn(r, make_float2(-kMagic, -kMagic));
        const float2 o = __ffma2_rn(q, make_float2(15.f, 15.f), make_float2(-e.x, -e.y));
        off = fmaxf(off, fmaxf(fabsf(o.x), fabsf(o.y)));
        n[j] = r.x;
        n[j + 1] = r.y;
    }
    if (off > 0.5f - 1e-5f) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            n[j] = __fadd_rn(fminf(fmaxf(__fdiv_rn(__fsub_rn(x[j], base), scale), 0.f), 15.f), kMagic);
    }
    // sum of (0x4b400000 + code_j) 16^j, less the constant's share 0x4b400000 (1 + 16 + 256) mod 2^32
    uint32_t word = 0u - 0x4b400000u * 273u;
#pragma unroll
    for (int j = 0; j < 8; ++j) word += __float_as_uint(n[j]) << (4 * j);
    return word;
}

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) kv4_append_kernel(const StoreParams p) {
    constexpr int kGroups = D / 64, kL = D / 16;
    const int l = threadIdx.x % kL;
    const RowOf r = row_of(p, kL);
    const T *src = (r.which ? static_cast<const T *>(p.v) + r.t * p.v_stride : static_cast<const T *>(p.k) + r.t * p.k_stride) +
                   r.h * D + 8 * l;
    pdl_wait();
    pdl_launch_dependents();
    const long long slot = slot_of(p, r);
    uint4 raw[2][sizeof(T) / 2];
    float x[2][8];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int i = 0; i < int(sizeof(T)) / 2; ++i)
            raw[b][i] = load(reinterpret_cast<const uint4 *>(src + b * 8 * kL) + i);
        Elems8<T>::unpack(raw[b], x[b]);
    }
    float2 ex = extremes<kGroups, kL>(raw, x, T());
    if (!(ex.x >= -kHalfMax) || !(ex.y >= -kHalfMax)) {  // the same for all lanes of the group
        bool odd = false;
        ex = make_float2(kHalfMax, kHalfMax);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            float &v = x[j / 8][j % 8];
            odd |= !(fabsf(v) <= kHalfMax);
            v = v != v ? 0.f : fminf(fmaxf(v, -kHalfMax), kHalfMax);
            ex.x = fminf(ex.x, v);
            ex.y = fminf(ex.y, -v);
        }
        if (odd && p.err && slot >= 0) atomicOr(p.err, SANTA_ERR_VALUE);
        unsigned group = 0;  // the lanes of this group in this warp
#pragma unroll
        for (int o = 0; o < kL; o += kGroups) group |= 1u << ((threadIdx.x & 31) / kL * kL + l % kGroups + o);
#pragma unroll
        for (int o = kGroups; o < kL; o <<= 1) {
            ex.x = fminf(ex.x, __shfl_xor_sync(group, ex.x, o));
            ex.y = fminf(ex.y, __shfl_xor_sync(group, ex.y, o));
        }
    }
    __syncwarp();
    const __half lo16 = __float2half_rn(ex.x);
    const float base = __half2float(lo16);
    const __half scale16 = __float2half_rn(__fmul_rn(__fsub_rn(-ex.y, base), 1.0f / 15.0f));
    const float scale = __half2float(scale16);
    const uint32_t word[2] = {codes_of(x[0], base, scale), codes_of(x[1], base, scale)};
    if (slot >= 0) {
        unsigned char *rec = p.kv4 + ((size_t)slot * p.Hkv + r.h) * kv4_record(D);
        uint32_t *words = reinterpret_cast<uint32_t *>(rec + r.which * (D / 2)) + l;
        words[0] = word[0];
        words[kL] = word[1];
        if (l < kGroups)
            reinterpret_cast<__half2 *>(rec + D + r.which * (D / 16))[l] = __halves2half2(scale16, lo16);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) kv4_read_kernel(const StoreParams p) {
    constexpr int kGroups = D / 64, kL = D / 16;
    const int l = threadIdx.x % kL;
    const RowOf r = row_of(p, kL);
    T *out = static_cast<T *>(r.which ? p.v_out : p.k_out);
    pdl_wait();
    pdl_launch_dependents();
    if (!r.live || !out) return;
    const long long slot = slot_of(p, r);
    uint32_t word[2] = {0u, 0u}, pair = 0u;
    if (slot >= 0) {
        const unsigned char *rec = p.kv4 + ((size_t)slot * p.Hkv + r.h) * kv4_record(D);
        const uint32_t *words = reinterpret_cast<const uint32_t *>(rec + r.which * (D / 2)) + l;
        word[0] = load(words);
        word[1] = load(words + kL);
        pair = load(reinterpret_cast<const uint32_t *>(rec + D + r.which * (D / 16)) + l % kGroups);
    }
    const float2 sm = __half22float2(*reinterpret_cast<const __half2 *>(&pair));
    // codes as fp16 subnormals, n 2^-24 and n 2^-20: the products with the scale stay exact
    const float2 m = make_float2(sm.y, sm.y), lo = make_float2(sm.x * 16777216.f, sm.x * 16777216.f),
                 hi = make_float2(sm.x * 1048576.f, sm.x * 1048576.f);
    T *row = out + ((size_t)r.t * p.Hkv + r.h) * D + 8 * l;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = word[b] >> (8 * i), c = w & 0x000f000fu, d = w & 0x00f000f0u;
            const float2 u = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&c)), lo, m);
            const float2 v = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&d)), hi, m);
            x[2 * i] = u.x, x[2 * i + 4] = u.y, x[2 * i + 1] = v.x, x[2 * i + 5] = v.y;
        }
        Elems8<T>::store(row + b * 8 * kL, x);
    }
}

template <typename K>
cudaError_t launch_rows(K kern, const StoreParams &p, int d, cudaStream_t stream) {
    const long long threads = (long long)p.tokens * 2 * p.Hkv * (d / 16);
    const long long ctas = (threads + kStoreThreads - 1) / kStoreThreads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_kernel(kern, dim3(unsigned(ctas)), dim3(kStoreThreads), 0, stream, true, 0, false, p);
}

}  // namespace

cudaError_t launch_kv4_append(const StoreParams &p, int dtype, int d, cudaStream_t stream) {
    if (dtype == SANTA_BF16)
        return launch_rows(d == 128 ? kv4_append_kernel<uint16_t, 128> : kv4_append_kernel<uint16_t, 64>, p, d, stream);
    return launch_rows(d == 128 ? kv4_append_kernel<float, 128> : kv4_append_kernel<float, 64>, p, d, stream);
}
cudaError_t launch_kv4_read(const StoreParams &p, int dtype, int d, cudaStream_t stream) {
    if (dtype == SANTA_BF16)
        return launch_rows(d == 128 ? kv4_read_kernel<uint16_t, 128> : kv4_read_kernel<uint16_t, 64>, p, d, stream);
    return launch_rows(d == 128 ? kv4_read_kernel<float, 128> : kv4_read_kernel<float, 64>, p, d, stream);
}

}  // namespace santa
