// santa_kv4_store.cu -- the 4-bit cache's append and read.
//
// A row (K or V of one token and KV head) is held by D / 8 lanes, one block of 8
// elements each; the blocks alternate between the row's D / 64 groups, so the lanes of a
// group are those with one value of l mod (D / 64).  Append: minimum and maximum over the
// group (three shuffles each), minimum and scale rounded to fp16 first, so that the codes
// are formed against the values that a reader will use:
//   code = rn((x - min) / scale) held to 0 .. 15.
// A lane's 8 codes are one 32-bit word of the record.  Every step is a single IEEE
// operation in fp32 (no fused multiply-add, division rounded to nearest), so the codes do
// not depend on how the kernel is compiled.
#include <cuda_fp16.h>

#include "santa_rows.cuh"
#include "santa_serving.h"

namespace santa {

namespace {

constexpr int kStoreThreads = 256;
constexpr float kHalfMax = 65504.f;

// Which row a thread's lanes take: the rows of a token are K of its KV heads, then V.
struct RowOf {
    long long t;
    int h, which, l;
    bool live;
};
template <int D>
__device__ __forceinline__ RowOf row_of(const StoreParams &p) {
    constexpr int kL = D / 8;
    const long long row = ((long long)blockIdx.x * kStoreThreads + threadIdx.x) / kL;
    const int per = 2 * p.Hkv;
    RowOf r;
    r.l = threadIdx.x % kL;
    r.t = row / per;
    r.live = r.t < p.tokens;
    if (!r.live) r.t = p.tokens - 1;
    const int i = int(row % per);
    r.which = i >= p.Hkv;
    r.h = i - r.which * p.Hkv;
    return r;
}

// The token's slot, -1 if it has none (padding, or beyond the cache: flagged).
__device__ __forceinline__ long long slot_of(const StoreParams &p, const RowOf &r) {
    long long slot = p.slot_map ? p.slot_map[r.t] : r.t;
    if (slot >= p.total_tokens) {
        if (p.err && r.live) atomicOr(p.err, SANTA_ERR_SLOT);
        slot = -1;
    }
    return slot < 0 ? -1 : slot;
}

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) kv4_append_kernel(const StoreParams p) {
    constexpr int kGroups = D / 64, kL = D / 8;
    const RowOf r = row_of<D>(p);
    pdl_wait();
    pdl_launch_dependents();
    const long long slot = slot_of(p, r);
    const T *src = r.which ? static_cast<const T *>(p.v) + r.t * p.v_stride : static_cast<const T *>(p.k) + r.t * p.k_stride;
    float x[8];
    Elems8<T>::load(src + r.h * D + 8 * r.l, x);
    bool odd = false;
    float lo = kHalfMax, hi = -kHalfMax;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        odd |= !(fabsf(x[j]) <= kHalfMax);
        x[j] = x[j] != x[j] ? 0.f : fminf(fmaxf(x[j], -kHalfMax), kHalfMax);
        lo = fminf(lo, x[j]);
        hi = fmaxf(hi, x[j]);
    }
#pragma unroll
    for (int o = kGroups; o < kL; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(kFull, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, o));
    }
    const __half lo16 = __float2half_rn(lo);
    const float base = __half2float(lo16);
    const __half scale16 = __float2half_rn(__fmul_rn(__fsub_rn(hi, base), 1.0f / 15.0f));
    const float scale = __half2float(scale16);
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float n = scale > 0.f ? rintf(__fdiv_rn(__fsub_rn(x[j], base), scale)) : 0.f;
        word |= uint32_t(fminf(fmaxf(n, 0.f), 15.f)) << (4 * j);
    }
    if (!r.live || slot < 0) return;
    if (odd && p.err) atomicOr(p.err, SANTA_ERR_VALUE);
    unsigned char *rec = p.kv4 + ((size_t)slot * p.Hkv + r.h) * kv4_record(D);
    reinterpret_cast<uint32_t *>(rec + r.which * (D / 2))[r.l] = word;
    if (r.l < kGroups)
        reinterpret_cast<__half2 *>(rec + D + r.which * (D / 16))[r.l] = __halves2half2(scale16, lo16);
}

template <typename T, int D>
__global__ void __launch_bounds__(kStoreThreads) kv4_read_kernel(const StoreParams p) {
    constexpr int kGroups = D / 64;
    const RowOf r = row_of<D>(p);
    pdl_wait();
    pdl_launch_dependents();
    T *dst = static_cast<T *>(r.which ? p.v_out : p.k_out);
    if (!r.live || !dst) return;
    const long long slot = slot_of(p, r);
    float x[8] = {};
    if (slot >= 0) {
        const unsigned char *rec = p.kv4 + ((size_t)slot * p.Hkv + r.h) * kv4_record(D);
        const uint32_t word = reinterpret_cast<const uint32_t *>(rec + r.which * (D / 2))[r.l];
        const float2 sm = __half22float2(reinterpret_cast<const __half2 *>(rec + D + r.which * (D / 16))[r.l % kGroups]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(sm.x, float((word >> (4 * j)) & 15u), sm.y);  // the product is exact
    }
    Elems8<T>::store(dst + ((size_t)r.t * p.Hkv + r.h) * D + 8 * r.l, x);
}

template <typename K>
cudaError_t launch_rows(K kern, const StoreParams &p, int d, cudaStream_t stream) {
    const long long threads = (long long)p.tokens * 2 * p.Hkv * (d / 8);
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
