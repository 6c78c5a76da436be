// santa_kv4_store.cu -- the 4-bit cache's append and read.
//
// A row (K or V of one token and KV head) is held by D / 8 lanes, one block of 8
// elements each; the blocks alternate between the row's D / 64 groups, so the lanes of a
// group are those with one value of l mod (D / 64).  Append: minimum and maximum over the
// group (three shuffles each), minimum and scale rounded to fp16 first, so that the codes
// are formed against the values that a reader will use:
//   code = rn((x - min) / scale) held to 0 .. 15.
// A lane's 8 codes are one 32-bit word of the record.  What is stored is defined by single
// IEEE operations in fp32 (no fused multiply-add, division rounded to nearest), so the codes
// do not depend on how the kernel is compiled.  The division itself is only done where it
// matters: with r an approximate reciprocal (2^-23), (x - min) r is off from the rounded
// quotient by less than 5 2^-24 of itself, 4.7e-6 for quotients below 15.5, so a result further
// than 1e-5 from the middle between two codes rounds as the quotient does.
//
// A prompt of 8191 tokens, 8 heads of 128, is 43 MB in and out for either direction (6.3 us at
// the copy rate).  Both are bound by instructions (211 and 110 per warp and row at first 295 and
// 149): 29 us for the two, at first 44.  What brought them down: one division per lane instead
// of one per row (a lane keeps its head and steps through tokens), packed minimum and maximum,
// no IEEE division, rounding and packing by the low bits of a large float, and codes read as
// fp16 subnormals.  One to four rows in flight per lane: 31.1, 29.6, 31.0, 31.3 us.
#include <cuda_fp16.h>

#include "santa_rows.cuh"
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kStoreThreads = 256;
constexpr int kMany = 2;  // rows of a lane in flight
constexpr float kHalfMax = 65504.f;

// The rows of a token are K of its KV heads, then V.  A lane row (D / 8 lanes) takes row
// `i` of the tokens t0, t0 + step, ...
struct RowOf {
    int t0, h, which;
    bool live;
};
__device__ __forceinline__ RowOf row_of(const StoreParams &p, int d8, int step) {
    const long long row = ((long long)blockIdx.x * kStoreThreads + threadIdx.x) / d8;
    const int per = 2 * p.Hkv;
    RowOf r;
    const long long t = row >> 31 ? row / per : (long long)(unsigned(row) / unsigned(per));
    r.live = t < step;
    r.t0 = r.live ? int(t) : 0;
    const int i = r.live ? int(row - t * per) : 0;
    r.which = i >= p.Hkv;
    r.h = i - r.which * p.Hkv;
    return r;
}

// Token t's slot, -1 if it has none (padding, beyond the last token, or beyond the cache: flagged).
__device__ __forceinline__ long long slot_of(const StoreParams &p, const RowOf &r, int t) {
    if (!r.live || t >= p.tokens) return -1;
    const long long slot = p.slot_map ? __ldg(p.slot_map + t) : t;
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
// (minimum, -maximum) of a group's elements, lane by lane and then over the lanes that hold
// the group (those whose index differs in bits >= log2 kGroups); NaN if there is one.
template <int kGroups, int kL>
__device__ __forceinline__ float2 extremes(const uint4 &raw, const float (&)[8], uint16_t) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    __nv_bfloat162 lo = *reinterpret_cast<const __nv_bfloat162 *>(&w[0]), hi = lo;
#pragma unroll
    for (int j = 1; j < 4; ++j) {
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
__device__ __forceinline__ float2 extremes(const uint4 &, const float (&x)[8], float) {
    float lo = x[0], hi = -x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) {
        lo = min_nan(lo, x[j]);
        hi = min_nan(hi, -x[j]);
    }
#pragma unroll
    for (int o = kGroups; o < kL; o <<= 1) {
        lo = min_nan(lo, __shfl_xor_sync(kFull, lo, o));
        hi = min_nan(hi, __shfl_xor_sync(kFull, hi, o));
    }
    return make_float2(lo, hi);
}

// The 8 codes of a lane, element j at bits 4 j.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float base, float scale) {
    constexpr float kMagic = 12582912.f;  // 1.5 2^23: adding it rounds to an integer in the low bits
    if (!(scale > 0.f)) return 0u;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    float n[8], off = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 d = __fadd2_rn(make_float2(x[j], x[j + 1]), make_float2(-base, -base));
        float2 q = __fmul2_rn(d, make_float2(inv, inv));
        q.x = fmaxf(fminf(q.x, 15.f), 0.f);  // the minimum's rounding can leave d < 0
        q.y = fmaxf(fminf(q.y, 15.f), 0.f);
        const float2 r = __fadd2_rn(q, make_float2(kMagic, kMagic));
        const float2 e = __fadd2_rn(__fadd2_rn(r, make_float2(-kMagic, -kMagic)), make_float2(-q.x, -q.y));
        off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
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

template <typename T, int D, int kRows>
__global__ void __launch_bounds__(kStoreThreads) kv4_append_kernel(const StoreParams p, int step) {
    constexpr int kGroups = D / 64, kL = D / 8;
    const int l = threadIdx.x % kL;
    const RowOf r = row_of(p, kL, step);
    const T *src = (r.which ? static_cast<const T *>(p.v) : static_cast<const T *>(p.k)) + r.h * D + 8 * l;
    const long long stride = r.which ? p.v_stride : p.k_stride;
    pdl_wait();
    pdl_launch_dependents();
    long long slot[kRows];
    uint4 raw[kRows][sizeof(T) / 2];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int t = r.t0 + k * step;
        slot[k] = slot_of(p, r, t);
        const uint4 *at = reinterpret_cast<const uint4 *>(src + min(t, p.tokens - 1) * stride);
#pragma unroll
        for (int i = 0; i < int(sizeof(T)) / 2; ++i) raw[k][i] = __ldg(at + i);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        float x[8];
        Elems8<T>::unpack(raw[k], x);
        float2 ex = extremes<kGroups, kL>(raw[k][0], x, T());
        if (!(ex.x >= -kHalfMax) || !(ex.y >= -kHalfMax)) {  // the same for all lanes of the group
            bool odd = false;
            ex = make_float2(kHalfMax, kHalfMax);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                odd |= !(fabsf(x[j]) <= kHalfMax);
                x[j] = x[j] != x[j] ? 0.f : fminf(fmaxf(x[j], -kHalfMax), kHalfMax);
                ex.x = fminf(ex.x, x[j]);
                ex.y = fminf(ex.y, -x[j]);
            }
            if (odd && p.err && slot[k] >= 0) atomicOr(p.err, SANTA_ERR_VALUE);
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
        const uint32_t word = codes_of(x, base, __half2float(scale16));
        if (slot[k] >= 0) {
            unsigned char *rec = p.kv4 + ((size_t)slot[k] * p.Hkv + r.h) * kv4_record(D);
            reinterpret_cast<uint32_t *>(rec + r.which * (D / 2))[l] = word;
            if (l < kGroups)
                reinterpret_cast<__half2 *>(rec + D + r.which * (D / 16))[l] = __halves2half2(scale16, lo16);
        }
    }
}

template <typename T, int D, int kRows>
__global__ void __launch_bounds__(kStoreThreads) kv4_read_kernel(const StoreParams p, int step) {
    constexpr int kGroups = D / 64, kL = D / 8;
    const int l = threadIdx.x % kL;
    const RowOf r = row_of(p, kL, step);
    T *out = static_cast<T *>(r.which ? p.v_out : p.k_out);
    pdl_wait();
    pdl_launch_dependents();
    if (!r.live || !out) return;
    long long slot[kRows];
    uint32_t word[kRows], pair[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) slot[k] = slot_of(p, r, r.t0 + k * step);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        word[k] = pair[k] = 0;
        if (slot[k] >= 0) {
            const unsigned char *rec = p.kv4 + ((size_t)slot[k] * p.Hkv + r.h) * kv4_record(D);
            word[k] = __ldg(reinterpret_cast<const uint32_t *>(rec + r.which * (D / 2)) + l);
            pair[k] = __ldg(reinterpret_cast<const uint32_t *>(rec + D + r.which * (D / 16)) + l % kGroups);
        }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int t = r.t0 + k * step;
        if (t >= p.tokens) break;
        const float2 sm = __half22float2(*reinterpret_cast<const __half2 *>(&pair[k]));
        // codes as fp16 subnormals, n 2^-24 and n 2^-20: the products with the scale stay exact
        const float2 m = make_float2(sm.y, sm.y), lo = make_float2(sm.x * 16777216.f, sm.x * 16777216.f),
                     hi = make_float2(sm.x * 1048576.f, sm.x * 1048576.f);
        float x[8];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = word[k] >> (8 * i), a = w & 0x000f000fu, b = w & 0x00f000f0u;
            const float2 u = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&a)), lo, m);
            const float2 v = __ffma2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&b)), hi, m);
            x[2 * i] = u.x, x[2 * i + 4] = u.y, x[2 * i + 1] = v.x, x[2 * i + 5] = v.y;
        }
        Elems8<T>::store(out + ((size_t)t * p.Hkv + r.h) * D + 8 * l, x);
    }
}

template <typename K>
cudaError_t launch_rows(K one, K many, const StoreParams &p, int d, cudaStream_t stream) {
    // a lane takes kMany tokens where they fill the GPU four times over all the same
    const long long lanes = 2LL * p.Hkv * (d / 8);
    const int per = p.tokens * lanes >= 152LL * 2048 * 4 ? kMany : 1;
    const int step = (p.tokens + per - 1) / per;
    const long long ctas = (step * lanes + kStoreThreads - 1) / kStoreThreads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_kernel(per == 1 ? one : many, dim3(unsigned(ctas)), dim3(kStoreThreads), 0, stream, true, 0, false, p,
                         step);
}

}  // namespace

#define SANTA_ROWS(kernel, T, D) launch_rows(kernel<T, D, 1>, kernel<T, D, kMany>, p, D, stream)
cudaError_t launch_kv4_append(const StoreParams &p, int dtype, int d, cudaStream_t stream) {
    if (dtype == SANTA_BF16)
        return d == 128 ? SANTA_ROWS(kv4_append_kernel, uint16_t, 128) : SANTA_ROWS(kv4_append_kernel, uint16_t, 64);
    return d == 128 ? SANTA_ROWS(kv4_append_kernel, float, 128) : SANTA_ROWS(kv4_append_kernel, float, 64);
}
cudaError_t launch_kv4_read(const StoreParams &p, int dtype, int d, cudaStream_t stream) {
    if (dtype == SANTA_BF16)
        return d == 128 ? SANTA_ROWS(kv4_read_kernel, uint16_t, 128) : SANTA_ROWS(kv4_read_kernel, uint16_t, 64);
    return d == 128 ? SANTA_ROWS(kv4_read_kernel, float, 128) : SANTA_ROWS(kv4_read_kernel, float, 64);
}
#undef SANTA_ROWS

}  // namespace santa
