// kvq_rope.cu -- rotary positions: the (cos, sin) table, and the rotation of a step's
// queries and keys fused with the quantisation of keys and values into the cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_dequant.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

// Angles p * freq_i in 64 bits: at position 10^6 a 32-bit product would already be off by
// 0.03 rad.  One thread per (position, pair); the table is made once per model.
__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ RopeTableParams p)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)p.n_pos * p.pairs) return;
    const int pair = (int)(i % p.pairs);
    const double angle = (double)(p.first_pos + i / p.pairs) * p.freq[pair];
    double s, c;
    sincos(angle, &s, &c);
    p.table[i] = make_float2((float)(c * p.gain), (float)(s * p.gain));
}

// A row is DH/4 lanes of four elements, so a warp handles 128/DH rows at a time and every
// load and store of a warp is one contiguous 128-element run.  The warp stays with one
// token: its lanes keep the (cos, sin) of their elements in registers and walk the token's
// query, key and value rows, kUnroll loads in flight.  `split` warps share a token so that
// a decode step's few tokens still fill the GPU.
constexpr int kUnroll = 4;

template <int DH>
__global__ void __launch_bounds__(256) rope_append_kernel(const __grid_constant__ RopeAppendParams p, int split)
{
    constexpr int LPR = DH / 4, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t token = w / split;
    if (token >= (int64_t)p.rows.batch * p.n_new) return;
    const int b = (int)(token / p.n_new), j = (int)(token % p.n_new);
    const int count = p.d_count ? min(p.d_count[b], p.n_new) : p.n_new;
    if (j >= count) return;
    const int first = p.d_pos[b];
    const int64_t pos = (int64_t)first + j;
    const int64_t rp = p.d_rope_pos ? p.d_rope_pos[token] : pos;
    if (rp < 0 || rp >= p.table_len) return;

    const int sub = lane / LPR, e0 = (lane % LPR) * 4;
    const int half = p.rot >> 1;
    // this lane's two or four (cos, sin) pairs; elements past rot pass through
    const bool turned = e0 < p.rot;
    const bool upper = !p.interleaved && e0 >= half;
    float c[4], s[4];
    if (turned) {
        const float2 *t = p.table + rp * half;
        if (p.interleaved) {
            const float4 a = *reinterpret_cast<const float4 *>(t + (e0 >> 1));
            c[0] = c[1] = a.x; s[0] = s[1] = a.y;
            c[2] = c[3] = a.z; s[2] = s[3] = a.w;
        } else {
            const float4 *q4 = reinterpret_cast<const float4 *>(t + (upper ? e0 - half : e0));
            const float4 a = q4[0], d = q4[1];
            c[0] = a.x; s[0] = a.y; c[1] = a.z; s[1] = a.w;
            c[2] = d.x; s[2] = d.y; c[3] = d.z; s[3] = d.w;
        }
    }
    const int partner = upper ? lane - half / 4 : lane + half / 4;

    // a token that a later token of this call overwrites in the ring is not stored
    bool keep = true;
    if (p.rows.window > 0 && pos >= p.rows.n_anchor)
        keep = pos + p.rows.window > (int64_t)first + count - 1;

    const int Hq = p.q_in.data ? p.n_q_heads : 0, Hkv = p.rows.heads;
    const int nq = (Hq + RPW - 1) / RPW, nk = (Hkv + RPW - 1) / RPW;
    const int total = nq + 2 * nk;
    for (int i0 = (int)(w % split); i0 < total; i0 += split * kUnroll) {
        float x[kUnroll][4];
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int i = i0 + u * split;
            const int kind = i < nq ? 0 : (i < nq + nk ? 1 : 2);   // query, key, value
            const int head = (i - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * RPW + sub;
            x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
            if (i < total && head < (kind == 0 ? Hq : Hkv)) {
                const RowsView &r = kind == 0 ? p.q_in : (kind == 1 ? p.k_in : p.v_in);
                load4(r.data, b * r.batch_stride + j * r.token_stride + (int64_t)head * DH + e0, p.dtype, x[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; u++) {
            const int i = i0 + u * split;
            if (i >= total) break;
            const int kind = i < nq ? 0 : (i < nq + nk ? 1 : 2);
            const int head = (i - (kind == 0 ? 0 : (kind == 1 ? nq : nq + nk))) * RPW + sub;
            const bool valid = head < (kind == 0 ? Hq : Hkv);
            float y[4] = {x[u][0], x[u][1], x[u][2], x[u][3]};
            if (kind != 2) {
                // every product and sum rounded on its own (no fused multiply-add), so that
                // codes and scales match an IEEE reference bit for bit
                float o[4];
#pragma unroll
                for (int e = 0; e < 4; e++)
                    o[e] = p.interleaved ? x[u][e ^ 1] : __shfl_sync(0xffffffffu, x[u][e], partner & 31);
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const bool second = p.interleaved ? (e & 1) : upper;
                        const float a = __fmul_rn(x[u][e], c[e]), d = __fmul_rn(o[e], s[e]);
                        y[e] = second ? __fadd_rn(a, d) : __fsub_rn(a, d);
                    }
                }
                if (kind == 0) {
                    if (valid)
                        store4(p.q_out.data, b * p.q_out.batch_stride + j * p.q_out.token_stride +
                               (int64_t)head * DH + e0, p.dtype, y);
                    continue;
                }
            }
            const CacheTensor &t = kind == 1 ? p.k : p.v;
            const int64_t row = valid && keep ? cache_row(p.rows, b, head, pos) : -1;
            __half *scales = t.bits == 16              ? nullptr
                             : p.fmt == KVQ_FMT_TENSOR ? t.scales
                                                       : t.scales + row * (DH / t.group) * scale_vals(p.fmt);
            quantize4(y, row >= 0, e0, t.bits, t.group, t.codes + row * (DH * t.bits / 8), scales, lane, p.fmt);
        }
    }
}

}  // namespace

cudaError_t launch_rope_table(const RopeTableParams &p, cudaStream_t stream)
{
    const int64_t n = (int64_t)p.n_pos * p.pairs;
    const int64_t blocks = (n + 255) / 256;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    (void)cudaGetLastError();
    rope_table_kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_rope_append(const RopeAppendParams &p, cudaStream_t stream)
{
    const int64_t tokens = (int64_t)p.rows.batch * p.n_new;
    const int rpw = 128 / p.dh;
    const int rows = ((p.q_in.data ? p.n_q_heads : 0) + rpw - 1) / rpw + 2 * ((p.rows.heads + rpw - 1) / rpw);
    // enough warps for 16 on every SM, as long as each keeps a row
    int64_t split = (148 * 16 + tokens - 1) / tokens;
    if (split > rows) split = rows;
    if (split < 1) split = 1;
    const int64_t blocks = (tokens * split + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    (void)cudaGetLastError();
    if (p.dh == 128)
        rope_append_kernel<128><<<(unsigned)blocks, 256, 0, stream>>>(p, (int)split);
    else
        rope_append_kernel<64><<<(unsigned)blocks, 256, 0, stream>>>(p, (int)split);
    return cudaGetLastError();
}

}  // namespace kvq
