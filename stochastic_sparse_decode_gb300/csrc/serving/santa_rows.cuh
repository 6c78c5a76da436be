// santa_rows.cuh -- rows of d elements held by d / 8 lanes, 8 consecutive elements each.
#pragma once

#include "santa_common.cuh"

namespace santa {

// 8 consecutive elements (16 bytes of bf16, 32 of fp32) as floats; storing rounds to nearest even.
template <typename T>
struct Elems8 {
    __device__ __forceinline__ static void load(const T *p, float (&x)[8]);
    __device__ __forceinline__ static void store(T *p, const float (&x)[8]);
};
template <>
struct Elems8<uint16_t> {
    __device__ __forceinline__ static void load(const uint16_t *p, float (&x)[8]) {
        const uint4 r = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    __device__ __forceinline__ static void store(uint16_t *p, const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Elems8<float> {
    __device__ __forceinline__ static void load(const float *p, float (&x)[8]) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ static void store(float *p, const float (&x)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

}  // namespace santa
