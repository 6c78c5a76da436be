// santa_rows.cuh -- rows of d elements held by d / 8 lanes, 8 consecutive elements each.
#pragma once

#include "santa_common.cuh"

namespace santa {

// 8 consecutive elements (16 bytes of bf16, 32 of fp32) as floats; storing rounds to nearest even.
template <typename T>
struct Elems8;
template <>
struct Elems8<uint16_t> {
    __device__ __forceinline__ static void unpack(const uint4 (&r)[1], float (&x)[8]) {
        const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
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
    __device__ __forceinline__ static void unpack(const uint4 (&r)[2], float (&x)[8]) {
        const uint32_t w[8] = {r[0].x, r[0].y, r[0].z, r[0].w, r[1].x, r[1].y, r[1].z, r[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ static void store(float *p, const float (&x)[8]) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// 4 consecutive elements (8 bytes of bf16, 16 of fp32), raw and as floats.
template <typename T>
struct Elems4;
template <>
struct Elems4<uint16_t> {
    using Raw = uint2;
    __device__ __forceinline__ static void unpack(const Raw &r, float (&x)[4]) {
        x[0] = bf16_lo(r.x), x[1] = bf16_hi(r.x), x[2] = bf16_lo(r.y), x[3] = bf16_hi(r.y);
    }
    __device__ __forceinline__ static Raw pack(const float (&x)[4]) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
    }
};
template <>
struct Elems4<float> {
    using Raw = float4;
    __device__ __forceinline__ static void unpack(const Raw &r, float (&x)[4]) {
        x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
    }
    __device__ __forceinline__ static Raw pack(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
};

}  // namespace santa
