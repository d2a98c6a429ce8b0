// kvq_dequant.cuh -- eight neighbouring elements of a cached row: codes as numbers, and
// the store of eight values.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/kvq.h"
#include "kvq_ptx.cuh"

namespace kvq {

template <int BITS>
struct Codes8;

template <>
struct Codes8<8> {
    uint2 w;
    __device__ __forceinline__ void load(const uint8_t *row, int chunk)
    {
        w = *reinterpret_cast<const uint2 *>(row + chunk * 8);
    }
    // signed, unsigned (zero-point) or e4m3 codes
    __device__ __forceinline__ void values(float (&x)[8], int fmt) const
    {
        const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (fmt == KVQ_FMT_E4M3) {
                const float2 a = unpack_half2(e4m3x2_to_half2(ww[i] & 0xffffu));
                const float2 b = unpack_half2(e4m3x2_to_half2(ww[i] >> 16));
                x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = b.x; x[4 * i + 3] = b.y;
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const uint32_t c = (ww[i] >> (8 * e)) & 0xffu;
                    x[4 * i + e] = fmt == KVQ_FMT_ASYM ? (float)c : (float)(int)(signed char)c;
                }
            }
        }
    }
};

template <>
struct Codes8<4> {
    uint32_t w;
    __device__ __forceinline__ void load(const uint8_t *row, int chunk)
    {
        w = *reinterpret_cast<const uint32_t *>(row + chunk * 4);
    }
    __device__ __forceinline__ void values(float (&x)[8], int) const
    {
#pragma unroll
        for (int e = 0; e < 8; e++) x[e] = (float)((int)(w << (28 - 4 * e)) >> 28);
    }
};

template <>
struct Codes8<16> {
    uint4 w;
    __device__ __forceinline__ void load(const uint8_t *row, int chunk)
    {
        w = *reinterpret_cast<const uint4 *>(row + chunk * 16);
    }
    __device__ __forceinline__ void values(float (&x)[8], int) const
    {
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 a = unpack_half2(ww[i]);
            x[2 * i] = a.x;
            x[2 * i + 1] = a.y;
        }
    }
};

// Four values at element idx (a multiple of 4), or two (a multiple of 2).
__device__ __forceinline__ void store4(void *base, int64_t idx, int dtype, const float (&x)[4])
{
    if (dtype == KVQ_F32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + idx) = make_float4(x[0], x[1], x[2], x[3]);
    } else if (dtype == KVQ_F16) {
        __half2 h[2] = {__floats2half2_rn(x[0], x[1]), __floats2half2_rn(x[2], x[3])};
        *reinterpret_cast<uint2 *>(static_cast<__half *>(base) + idx) = *reinterpret_cast<uint2 *>(h);
    } else {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x[0], x[1]), __floats2bfloat162_rn(x[2], x[3])};
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(base) + idx) = *reinterpret_cast<uint2 *>(h);
    }
}

__device__ __forceinline__ void store2(void *base, int64_t idx, int dtype, const float (&x)[2])
{
    if (dtype == KVQ_F32)
        *reinterpret_cast<float2 *>(static_cast<float *>(base) + idx) = make_float2(x[0], x[1]);
    else if (dtype == KVQ_F16)
        *reinterpret_cast<__half2 *>(static_cast<__half *>(base) + idx) = __floats2half2_rn(x[0], x[1]);
    else
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(base) + idx) = __floats2bfloat162_rn(x[0], x[1]);
}

// Eight values at element idx (a multiple of 8) of an array of dtype.
__device__ __forceinline__ void store8(void *base, int64_t idx, int dtype, const float (&x)[8])
{
    if (dtype == KVQ_F32) {
        float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(base) + idx);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
        return;
    }
    uint4 w;
    uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (dtype == KVQ_F16) {
            ww[i] = pack_half2(x[2 * i], x[2 * i + 1]);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            ww[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + idx) = w;
}

}  // namespace kvq
