// kvq_rope.cu -- rotary positions: the (cos, sin) table, and the rotation of a step's
// queries and keys fused with the quantisation of keys and values into the cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_dequant.cuh"
#include "kvq_internal.h"
#include "kvq_ptx.cuh"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

// Angles p * freq_i in 64 bits: at position 10^6 a 32-bit product would already be off by
// 0.03 rad.  One thread per (position, pair); the table is made once per model.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)p.n_pos * p.pairs) return;
    const int pair = (int)(i % p.pairs);
    const double angle = (double)(p.first_pos + i / p.pairs) * p.freq[pair];
    double s, c;
    sincos(angle, &s, &c);
    p.table[i] = make_float2((float)(c * p.gain), (float)(s * p.gain));
}

// Integer code of x at scale s (inv = 1 / s to within 2^-22): rne of the IEEE quotient x / s.
// The product with the inverse is at most 2^-21 of |x / s| <= 2^8 off the quotient, so away
// from the midpoints between integers both round alike; `near` reports the rest (one element in
// 2500), for which the caller divides.
__device__ __forceinline__ float code_of(float x, float inv, bool &near)
{
    const float y = x * inv, n = rintf(y);
    near |= fabsf(fabsf(y - n) - 0.5f) < 2e-4f;
    return n;
}

// Quantise a row that LPR lanes hold, lane t elements 4t .. 4t+3 (v[0]) and DH/2 + 4t .. (v[1]),
// as quantize4 does: the same codes and scales bit for bit.
template <int DH>
__device__ __forceinline__ void quantize_row8(const float (&v)[2][4], bool active, int t, int bits, int group, int fmt,
                                              uint8_t *codes, __half *scales)
{
    constexpr int LPR = DH / 8;
    if (bits == 16) {
        if (!active) return;
#pragma unroll
        for (int h = 0; h < 2; h++)
            *reinterpret_cast<uint2 *>(codes + (h * DH / 2 + 4 * t) * 2) =
                make_uint2(pack_half2(v[h][0], v[h][1]), pack_half2(v[h][2], v[h][3]));
        return;
    }
    // lanes of a group's half, and whether both halves are one group
    const bool joint = group == DH;
    const int span = min(group >> 2, LPR);
    float lo[2], hi[2];                          // per half: least and largest, or largest magnitude
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if (fmt == KVQ_FMT_ASYM) {
            lo[h] = fminf(fminf(fminf(v[h][0], v[h][1]), fminf(v[h][2], v[h][3])), 0.f);
            hi[h] = fmaxf(fmaxf(fmaxf(v[h][0], v[h][1]), fmaxf(v[h][2], v[h][3])), 0.f);
        } else {
            lo[h] = 0.f;
            hi[h] = fmaxf(fmaxf(fabsf(v[h][0]), fabsf(v[h][1])), fmaxf(fabsf(v[h][2]), fabsf(v[h][3])));
        }
    }
    if (joint) {
        lo[0] = fminf(lo[0], lo[1]);
        hi[0] = fmaxf(hi[0], hi[1]);
    }
    if (fmt != KVQ_FMT_TENSOR) {
#pragma unroll 1
        for (int off = 1; off < span; off <<= 1) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (h == 1 && joint) break;
                hi[h] = fmaxf(hi[h], __shfl_xor_sync(0xffffffffu, hi[h], off));
                if (fmt == KVQ_FMT_ASYM) lo[h] = fminf(lo[h], __shfl_xor_sync(0xffffffffu, lo[h], off));
            }
        }
    }
    if (joint) {
        lo[1] = lo[0];
        hi[1] = hi[0];
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int e0 = h * DH / 2 + 4 * t;
        const int qmax = bits == 4 ? 7 : 127;
        __half s16;
        if (fmt == KVQ_FMT_TENSOR) {
            s16 = scales[0];
        } else {
            const float top = fmt == KVQ_FMT_ASYM ? __fsub_rn(hi[h], lo[h]) : hi[h];
            const float by = fmt == KVQ_FMT_ASYM ? 255.f : fmt == KVQ_FMT_E4M3 ? 448.f : (float)qmax;
            s16 = __float2half_rn(__fdiv_rn(top, by));
            if (__half_as_ushort(s16) == 0x7c00u) s16 = __ushort_as_half(0x7bffu);
        }
        const float s = __half2float(s16);
        const bool zero = s == 0.f;
        int z = 0;
        if (fmt == KVQ_FMT_ASYM && !zero) z = max(0, min(255, __float2int_rn(__fdiv_rn(-lo[h], s))));
        uint32_t w = 0;
        if (fmt == KVQ_FMT_E4M3) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                w |= (zero ? 0u : (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(v[h][e], s), __NV_SATFINITE, __NV_E4M3)) << (8 * e);
        } else {
            const float inv = zero ? 0.f : __fdividef(1.f, s);
            // (a scale far below the values, or above 2^126, leaves the inverse's range)
            bool near = !(inv > 0.f) || fmt == KVQ_FMT_TENSOR;
            float n[4];
#pragma unroll
            for (int e = 0; e < 4; e++) n[e] = code_of(v[h][e], inv, near);
            if (near && !zero) {
#pragma unroll
                for (int e = 0; e < 4; e++) n[e] = rintf(__fdiv_rn(v[h][e], s));
            }
            const float least = fmt == KVQ_FMT_ASYM ? 0.f : (float)-qmax, most = fmt == KVQ_FMT_ASYM ? 255.f : (float)qmax;
            uint32_t q[4];
#pragma unroll
            for (int e = 0; e < 4; e++) q[e] = zero ? 0u : (uint32_t)(int)fminf(fmaxf(n[e] + (float)z, least), most);
            if (bits == 4)
                w = (q[0] & 15u) | (q[1] & 15u) << 4 | (q[2] & 15u) << 8 | (q[3] & 15u) << 12;
            else
                w = (q[0] & 255u) | (q[1] & 255u) << 8 | (q[2] & 255u) << 16 | q[3] << 24;
        }
        if (!active) continue;
        if (bits == 4)
            *reinterpret_cast<uint16_t *>(codes + e0 / 2) = (uint16_t)w;
        else
            *reinterpret_cast<uint32_t *>(codes + e0) = w;
        if (fmt != KVQ_FMT_TENSOR && t % span == 0 && !(h == 1 && joint)) {
            if (fmt == KVQ_FMT_ASYM)
                reinterpret_cast<__half2 *>(scales)[e0 / group] = __halves2half2(s16, __int2half_rn(z));
            else
                scales[e0 / group] = s16;
        }
    }
}

// A row is DH/8 lanes of eight elements, four in each half of the row, so that a warp's loads
// and stores are whole runs and the pairs of a fully rotated half layout meet in one lane.  A
// warp stays with one token: its lanes keep the (cos, sin) of their elements in registers and
// walk the token's query, key and value rows, kUnroll of them in flight.  `split` warps share
// a token so that a decode step's few tokens still fill the GPU.
// MODE 0: half layout, whole row; 1: interleaved; 2: half layout, part of the row (partners
// come by shuffles).
constexpr int kUnroll = 4;

template <int DH, int MODE>
__global__ void __launch_bounds__(256) rope_append_kernel(const __grid_constant__ RopeAppendParams p, int split)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int LPR = DH / 8, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t token = w / split;
    if (token >= (int64_t)p.rows.batch * p.n_new) return;
    const int b = (int)(token / p.n_new), j = (int)(token - (int64_t)b * p.n_new);
    const int count = p.d_count ? min(p.d_count[b], p.n_new) : p.n_new;
    if (j >= count) return;
    const int first = p.d_pos[b];
    const int64_t pos = (int64_t)first + j;
    const int64_t rp = p.d_rope_pos ? p.d_rope_pos[token] : pos;
    if (rp < 0 || rp >= p.table_len) return;

    const int sub = lane / LPR, t = lane % LPR;
    const int half = p.rot >> 1;
    // (cos, sin) of this lane's elements, and where an element's partner is
    float c[2][4], s[2][4];
    bool turned[2], upper[2];
    int from[2];                                 // MODE 2: lane and half (bit 5) of the partner chunk
    const float2 *row = p.table + rp * half;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int e0 = h * DH / 2 + 4 * t;
        turned[h] = e0 < p.rot;
        upper[h] = MODE == 0 ? h == 1 : MODE == 2 && e0 >= half;
        const int partner = (upper[h] ? e0 - half : e0 + half) >> 2;      // chunk of four elements
        from[h] = (sub * LPR + partner % LPR) | (partner / LPR) << 5;
        if (MODE == 0 && h == 1) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                c[1][e] = c[0][e];
                s[1][e] = s[0][e];
            }
        } else if (turned[h]) {
            if (MODE == 1) {
                const float4 a = *reinterpret_cast<const float4 *>(row + (e0 >> 1));
                c[h][0] = c[h][1] = a.x; s[h][0] = s[h][1] = a.y;
                c[h][2] = c[h][3] = a.z; s[h][2] = s[h][3] = a.w;
            } else {
                const float4 *q4 = reinterpret_cast<const float4 *>(row + (upper[h] ? e0 - half : e0));
                const float4 a = q4[0], d = q4[1];
                c[h][0] = a.x; s[h][0] = a.y; c[h][1] = a.z; s[h][1] = a.w;
                c[h][2] = d.x; s[h][2] = d.y; c[h][3] = d.z; s[h][3] = d.w;
            }
        }
    }

    // a token that a later token of this call overwrites in the ring is not stored
    bool keep = true;
    if (p.rows.window > 0 && pos >= p.rows.n_anchor)
        keep = pos + p.rows.window > (int64_t)first + count - 1;
    const int64_t row0 = keep ? cache_row(p.rows, b, 0, pos) : -1;       // head 0's row; heads lie apart by:
    const int64_t head_rows = p.rows.block_table ? kPageTokens : p.rows.cap;

    const int Hq = p.q_in.data ? p.n_q_heads : 0, Hkv = p.rows.heads;
    const int nq = (Hq + RPW - 1) / RPW, nk = (Hkv + RPW - 1) / RPW;
    const int total = nq + 2 * nk;
#pragma unroll 1
    for (int i0 = (int)(w - token * split); i0 < total; i0 += split * kUnroll) {
        float x[kUnroll][2][4];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int i = i0 + u * split;
            const int kind = i < nq ? 0 : (i < nq + nk ? 1 : 2);   // query, key, value
            const int head = (i - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * RPW + sub;
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int e = 0; e < 4; e++) x[u][h][e] = 0.f;
            if (i < total && head < (kind == 0 ? Hq : Hkv)) {
                const RowsView &r = kind == 0 ? p.q_in : (kind == 1 ? p.k_in : p.v_in);
                const int64_t at = b * r.batch_stride + j * r.token_stride + (int64_t)head * DH + 4 * t;
                load4(r.data, at, p.dtype, x[u][0]);
                load4(r.data, at + DH / 2, p.dtype, x[u][1]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int i = i0 + u * split;
            if (i >= total) break;
            const int kind = i < nq ? 0 : (i < nq + nk ? 1 : 2);
            const int head = (i - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * RPW + sub;
            const bool valid = head < (kind == 0 ? Hq : Hkv);
            float y[2][4];
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int e = 0; e < 4; e++) y[h][e] = x[u][h][e];
            if (kind != 2) {
                // every product and sum rounded on its own (no fused multiply-add), so that
                // codes and scales match an IEEE reference bit for bit
#pragma unroll
                for (int h = 0; h < 2; h++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        float o;
                        if (MODE == 0) {
                            o = x[u][h ^ 1][e];
                        } else if (MODE == 1) {
                            o = x[u][h][e ^ 1];
                        } else {
                            const float o0 = __shfl_sync(0xffffffffu, x[u][0][e], from[h] & 31);
                            const float o1 = __shfl_sync(0xffffffffu, x[u][1][e], from[h] & 31);
                            o = from[h] & 32 ? o1 : o0;
                        }
                        if (MODE == 0 || turned[h]) {
                            const bool second = MODE == 1 ? (e & 1) : upper[h];
                            const float a = __fmul_rn(x[u][h][e], c[h][e]), d = __fmul_rn(o, s[h][e]);
                            y[h][e] = second ? __fadd_rn(a, d) : __fsub_rn(a, d);
                        }
                    }
                if (kind == 0) {
                    if (valid) {
                        const int64_t at = b * p.q_out.batch_stride + j * p.q_out.token_stride + (int64_t)head * DH + 4 * t;
                        store4(p.q_out.data, at, p.dtype, y[0]);
                        store4(p.q_out.data, at + DH / 2, p.dtype, y[1]);
                    }
                    continue;
                }
            }
            const CacheTensor &ten = kind == 1 ? p.k : p.v;
            const bool active = valid && row0 >= 0;
            const int64_t cr = active ? row0 + head * head_rows : 0;
            quantize_row8<DH>(y, active, t, ten.bits, ten.group, p.fmt, ten.codes + cr * (DH * ten.bits / 8),
                              ten.bits == 16 || p.fmt == KVQ_FMT_TENSOR
                                  ? ten.scales : ten.scales + cr * (DH / ten.group) * scale_vals(p.fmt));
        }
    }
}

template <int DH>
cudaError_t launch_append_dh(const RopeAppendParams &p, unsigned blocks, int split, cudaStream_t stream)
{
    if (p.interleaved) return launch_dependent(rope_append_kernel<DH, 1>, blocks, 256, 0, stream, p, split);
    if (p.rot == DH) return launch_dependent(rope_append_kernel<DH, 0>, blocks, 256, 0, stream, p, split);
    return launch_dependent(rope_append_kernel<DH, 2>, blocks, 256, 0, stream, p, split);
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams &p, cudaStream_t stream)
{
    const int64_t n = (int64_t)p.n_pos * p.pairs;
    const int64_t blocks = (n + 255) / 256;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(rope_table_kernel, (unsigned)blocks, 256, 0, stream, p);
}

cudaError_t launch_rope_append(const RopeAppendParams &p, cudaStream_t stream)
{
    const int64_t tokens = (int64_t)p.rows.batch * p.n_new;
    const int rpw = 256 / p.dh;
    const int rows = ((p.q_in.data ? p.n_q_heads : 0) + rpw - 1) / rpw + 2 * ((p.rows.heads + rpw - 1) / rpw);
    // enough warps for 32 on every SM, as long as each keeps a row
    int64_t split = (148 * 32 + tokens - 1) / tokens;
    if (split > rows) split = rows;
    if (split < 1) split = 1;
    const int64_t blocks = (tokens * split + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return p.dh == 128 ? launch_append_dh<128>(p, (unsigned)blocks, (int)split, stream)
                       : launch_append_dh<64>(p, (unsigned)blocks, (int)split, stream);
}

}  // namespace kvq
