// kvq_dequant.cuh -- eight neighbouring codes of a cached row as f16 numbers, and stores of
// a few values in any of the output types.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/kvq.h"
#include "kvq_ptx.cuh"

namespace kvq {

enum { K_INT8, K_INT4, K_E4M3, K_ASYM, K_F16 };

__device__ __forceinline__ int kind_of(int bits, int fmt)
{
    return bits == 4 ? K_INT4 : bits == 16 ? K_F16 : fmt == KVQ_FMT_E4M3 ? K_E4M3 : fmt == KVQ_FMT_ASYM ? K_ASYM : K_INT8;
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2_u32(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

template <int KIND>
struct Raw;
template <> struct Raw<K_INT8> { uint2 w; static constexpr int BYTES = 8; };
template <> struct Raw<K_ASYM> { uint2 w; static constexpr int BYTES = 8; };
template <> struct Raw<K_E4M3> { uint2 w; static constexpr int BYTES = 8; };
template <> struct Raw<K_INT4> { uint32_t w; static constexpr int BYTES = 4; };
template <> struct Raw<K_F16> { uint4 w; static constexpr int BYTES = 16; };

// Eight codes as f16, element pairs in the words' low and high halves.  Bytes become f16 by
// putting them under the exponent of 1024 (0x64 in the high byte) and subtracting.
template <int KIND>
__device__ __forceinline__ void codes_f16(const Raw<KIND> &r, uint32_t zero, uint32_t (&h)[4])
{
    if constexpr (KIND == K_INT8 || KIND == K_ASYM) {
        const uint32_t flip = KIND == K_INT8 ? 0x80808080u : 0u;
        const uint32_t base = KIND == K_INT8 ? 0x64806480u : zero;   // 1024 + 128, or 1024 + zero-point
        const uint32_t a = r.w.x ^ flip, b = r.w.y ^ flip;
        h[0] = hsub2_u32(prmt(a, 0x64646464u, 0x4140), base);
        h[1] = hsub2_u32(prmt(a, 0x64646464u, 0x4342), base);
        h[2] = hsub2_u32(prmt(b, 0x64646464u, 0x4140), base);
        h[3] = hsub2_u32(prmt(b, 0x64646464u, 0x4342), base);
    } else if constexpr (KIND == K_INT4) {
        // byte k twice; the low nibble stays (1024 + n), the high one is at 16 n (1024 + 16 n);
        // the flipped sign bit adds 8 to each, and the multiply-add removes offset and factor
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint32_t x = prmt(r.w, 0u, (4u << 12) | ((uint32_t)k << 8) | (4u << 4) | (uint32_t)k);
            h[k] = hfma2_u32(and_xor(x, 0x00F0000Fu, 0x64806408u), 0x2C003C00u, 0xD480E408u);
        }
    } else if constexpr (KIND == K_E4M3) {
        h[0] = e4m3x2_to_half2(r.w.x & 0xffffu);
        h[1] = e4m3x2_to_half2(r.w.x >> 16);
        h[2] = e4m3x2_to_half2(r.w.y & 0xffffu);
        h[3] = e4m3x2_to_half2(r.w.y >> 16);
    } else {
        h[0] = r.w.x; h[1] = r.w.y; h[2] = r.w.z; h[3] = r.w.w;
    }
}

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
