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
// 0.03 rad.  One thread per (position, pair), bound by the 64-bit sine and cosine: 131072
// positions of 64 pairs take 72 us.  The table is made once per model.
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

// Integer codes of eight elements at scale s (inv = 1 / s to within 2^-22), as the low bytes of
// t: rne of the IEEE quotients x / s, plus z, clamped.  x * inv + 1.5 * 2^23 rounds the product
// with the inverse to an integer; it is at most 2^-13 off the quotient (|x / s| < 2^8, above
// that both are clamped), so away from the midpoints between integers both round alike.  Near
// one (an element in 2500 is), and where an element or the scale is no finite number, the lane
// divides and converts as quantize_row does.
__device__ __forceinline__ void codes_of(const float (&x)[8], float s, float inv, int z, int least, int most,
                                         uint32_t (&t)[8])
{
    constexpr float kRound = 12582912.f;
    // (a scale far below the values, a negative or an infinite one leave the inverse's range)
    bool far = inv > 0.f;
    float n[8];
#pragma unroll
    for (int e = 0; e < 8; e++) {
        n[e] = fmaf(x[e], inv, kRound);
        far &= fabsf(fmaf(x[e], inv, kRound - n[e])) <= 0.4998f;
    }
    if (!far && s != 0.f) {
#pragma unroll
        for (int e = 0; e < 8; e++)      // (the sum wraps around where the quotient has saturated, as there)
            t[e] = (uint32_t)max(least, min(most, (int)((uint32_t)__float2int_rn(__fdiv_rn(x[e], s)) + (uint32_t)z)));
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; e++)
        t[e] = s == 0.f ? 0u : __float_as_uint(fminf(fmaxf(n[e] + (float)z, kRound + (float)least), kRound + (float)most));
}

// Quantise a row that LPR lanes hold, lane t elements 8t .. 8t+7 (v[0]) and DH/2 + 8t .. (v[1]),
// as quantize_row does: the same codes and scales bit for bit.
template <int DH>
__device__ __forceinline__ void quantize_row16(const float (&v)[2][8], bool active, int t, int bits, int gshift, int fmt,
                                               uint8_t *codes, __half *scales)
{
    constexpr int LPR = DH / 16;
    if (bits == 16) {
        if (!active) return;
#pragma unroll
        for (int h = 0; h < 2; h++)
            *reinterpret_cast<uint4 *>(codes + (h * DH / 2 + 8 * t) * 2) =
                make_uint4(pack_half2(v[h][0], v[h][1]), pack_half2(v[h][2], v[h][3]), pack_half2(v[h][4], v[h][5]),
                           pack_half2(v[h][6], v[h][7]));
        return;
    }
    // lanes of a group's half, and whether both halves are one group
    const bool joint = (1 << gshift) == DH;
    const int span = min(1 << (gshift - 3), LPR);
    float lo[2], hi[2];                          // per half: least and largest, or largest magnitude
#pragma unroll
    for (int h = 0; h < 2; h++) {
        lo[h] = 0.f;
        // (maxima pass over NaN; a group of nothing else has a NaN scale)
        hi[h] = fmt == KVQ_FMT_ASYM ? 0.f : fabsf(v[h][0]);
        if (fmt == KVQ_FMT_ASYM) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                lo[h] = fminf(lo[h], v[h][e]);
                hi[h] = fmaxf(hi[h], v[h][e]);
            }
        } else {
#pragma unroll
            for (int e = 1; e < 8; e++) hi[h] = fmaxf(hi[h], fabsf(v[h][e]));
        }
    }
    if (joint) {
        lo[0] = fminf(lo[0], lo[1]);
        hi[0] = fmaxf(hi[0], hi[1]);
    }
    if (fmt != KVQ_FMT_TENSOR) {
#pragma unroll
        for (int off = 1; off < LPR; off <<= 1) {
            if (off >= span) break;
#pragma unroll
            for (int h = 0; h < 2; h++) {
                if (h == 1 && joint) break;
                hi[h] = fmaxf(hi[h], __shfl_xor_sync(0xffffffffu, hi[h], off));
                if (fmt == KVQ_FMT_ASYM) lo[h] = fminf(lo[h], __shfl_xor_sync(0xffffffffu, lo[h], off));
            }
        }
    }
    const float qmax = bits == 4 ? 7.f : 127.f;
    __half s16;
    float s = 0.f, inv = 0.f;
    int z = 0;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int e0 = h * DH / 2 + 8 * t;
        if (h == 0 || !joint) {
            if (fmt == KVQ_FMT_TENSOR) {
                s16 = scales[0];
            } else {
                const float top = fmt == KVQ_FMT_ASYM ? __fsub_rn(hi[h], lo[h]) : hi[h];
                const float by = fmt == KVQ_FMT_ASYM ? 255.f : fmt == KVQ_FMT_E4M3 ? 448.f : qmax;
                s16 = __float2half_rn(__fdiv_rn(top, by));
                if (__half_as_ushort(s16) == 0x7c00u) s16 = __ushort_as_half(0x7bffu);
            }
            s = __half2float(s16);
            z = fmt == KVQ_FMT_ASYM && s != 0.f ? max(0, min(255, __float2int_rn(__fdiv_rn(-lo[h], s)))) : 0;
            inv = s == 0.f ? 0.f : __fdividef(1.f, s);
        }
        uint32_t w[2];
        if (fmt == KVQ_FMT_E4M3) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                w[k] = 0;
#pragma unroll
                for (int e = 0; e < 4; e++)
                    w[k] |= (s == 0.f ? 0u : (uint32_t)__nv_cvt_float_to_fp8(__fdiv_rn(v[h][4 * k + e], s), __NV_SATFINITE,
                                                                              __NV_E4M3)) << (8 * e);
            }
        } else {
            uint32_t q[8];
            if (fmt == KVQ_FMT_ASYM)
                codes_of(v[h], s, inv, z, 0, 255, q);
            else
                codes_of(v[h], s, inv, 0, -(int)qmax, (int)qmax, q);
#pragma unroll
            for (int k = 0; k < 2; k++)
                w[k] = __byte_perm(__byte_perm(q[4 * k], q[4 * k + 1], 0x0040), __byte_perm(q[4 * k + 2], q[4 * k + 3], 0x0040),
                                   0x5410);
        }
        if (!active) continue;
        if (bits == 4) {
            // eight codes, one a byte, to eight nibbles
#pragma unroll
            for (int k = 0; k < 2; k++) {
                w[k] &= 0x0f0f0f0fu;
                w[k] |= w[k] >> 4;
            }
            *reinterpret_cast<uint32_t *>(codes + e0 / 2) =
                __byte_perm(w[0], w[1], 0x6420);
        } else {
            *reinterpret_cast<uint2 *>(codes + e0) = make_uint2(w[0], w[1]);
        }
        if (fmt != KVQ_FMT_TENSOR && (t & (span - 1)) == 0 && !(h == 1 && joint)) {
            if (fmt == KVQ_FMT_ASYM)
                reinterpret_cast<__half2 *>(scales)[e0 >> gshift] = __halves2half2(s16, __int2half_rn(z));
            else
                scales[e0 >> gshift] = s16;
        }
    }
}

// A lane's 16 elements as they lie in memory: eight of each half of the row.
template <int DT>
struct Raw16 {
    static constexpr int N = DT == KVQ_F32 ? 2 : 1;
    uint4 u[2][N];
    template <int DH>
    __device__ __forceinline__ void load(const void *base, int64_t idx)
    {
        constexpr int B = DT == KVQ_F32 ? 4 : 2;
        const uint8_t *src = static_cast<const uint8_t *>(base) + idx * B;
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int k = 0; k < N; k++) u[h][k] = *reinterpret_cast<const uint4 *>(src + h * (DH / 2) * B + 16 * k);
    }
    __device__ __forceinline__ void values(float (&x)[2][8]) const
    {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int k = 0; k < N; k++) {
                const uint32_t w[4] = {u[h][k].x, u[h][k].y, u[h][k].z, u[h][k].w};
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    if constexpr (DT == KVQ_F32) {
                        x[h][4 * k + q] = __uint_as_float(w[q]);
                    } else if constexpr (DT == KVQ_F16) {
                        const float2 f = unpack_half2(w[q]);
                        x[h][2 * q] = f.x;
                        x[h][2 * q + 1] = f.y;
                    } else {
                        x[h][2 * q] = __uint_as_float(w[q] << 16);
                        x[h][2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
                    }
                }
            }
    }
};

// A row is DH/16 lanes of 16 elements, eight in each half of the row, so that a warp's loads
// and stores are whole 16-byte runs and the pairs of a fully rotated half layout meet in one
// lane.  A warp stays with one token: its lanes keep the (cos, sin) of their elements in
// registers and walk the token's query, key and value rows.  `split` warps share a token so
// that a decode step's few tokens still fill the GPU.
// HBM bounds it in theory, latency and instructions in practice: 2 x 4096 tokens of 32 query
// and 8 KV heads of 128, bf16 in, INT8 in the cache: 41.7 us, 4.4 TB/s (with eight elements a
// lane, run-time types and divisions by the group size it took 7200 instructions a token and
// three times as long); a step of 64 tokens 3.2 us.
// MODE 0: half layout, whole row; 1: interleaved; 2: half layout, part of the row (partners
// are read a second time, from the cache line that a neighbour has just fetched).
template <int DH, int MODE>
struct Turn {
    static constexpr int NC = MODE == 2 ? 16 : 8;
    float c[NC], s[NC];                          // MODE 0: of both halves; 1: of the pairs; 2: of the elements
    bool turned[2];                              // MODE 1, 2: whether the half's elements turn
    int rot, t;

    __device__ __forceinline__ void load(const float2 *row, int rot_, int t_)
    {
        rot = rot_;
        t = t_;
        const int half = rot >> 1;
#pragma unroll
        for (int h = 0; h < 2; h++) turned[h] = MODE == 0 || h * DH / 2 + 8 * t < rot;
#pragma unroll
        for (int k = 0; k < NC / 4; k++) {
            // four pairs: of elements e .. e+3 (or of their partners), or 2e .. 2e+7
            int at;
            bool live = true;
            if (MODE == 0) {
                at = 8 * t + 4 * k;
            } else if (MODE == 1) {
                at = (k * DH / 2 + 8 * t) >> 1;
                live = turned[k];
            } else {
                const int e = (k >> 1) * DH / 2 + 8 * t + 4 * (k & 1);
                at = e < half ? e : e - half;
                live = turned[k >> 1];
            }
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
            if (live) {
                a = reinterpret_cast<const float4 *>(row + at)[0];
                d = reinterpret_cast<const float4 *>(row + at)[1];
            }
            c[4 * k] = a.x; s[4 * k] = a.y; c[4 * k + 1] = a.z; s[4 * k + 1] = a.w;
            c[4 * k + 2] = d.x; s[4 * k + 2] = d.y; c[4 * k + 3] = d.z; s[4 * k + 3] = d.w;
        }
    }
    // The lane's elements x of the row whose element 0 is src[at], turned.  Every product and
    // sum is rounded on its own (no fused multiply-add), so that codes and scales match an IEEE
    // reference bit for bit.
    template <int DT>
    __device__ __forceinline__ void apply(float (&x)[2][8], const void *src, int64_t at) const
    {
        if constexpr (MODE == 0) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float a = x[0][e], b = x[1][e];
                x[0][e] = __fsub_rn(__fmul_rn(a, c[e]), __fmul_rn(b, s[e]));
                x[1][e] = __fadd_rn(__fmul_rn(b, c[e]), __fmul_rn(a, s[e]));
            }
        } else if constexpr (MODE == 1) {
#pragma unroll
            for (int h = 0; h < 2; h++)
                if (turned[h])
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const float a = x[h][2 * e], b = x[h][2 * e + 1], ce = c[4 * h + e], se = s[4 * h + e];
                        x[h][2 * e] = __fsub_rn(__fmul_rn(a, ce), __fmul_rn(b, se));
                        x[h][2 * e + 1] = __fadd_rn(__fmul_rn(b, ce), __fmul_rn(a, se));
                    }
        } else {
            const int half = rot >> 1;
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const int h = k >> 1, e = h * DH / 2 + 8 * t + 4 * (k & 1);
                const bool upper = e >= half;
                if (turned[h]) {
                    float o[4];
                    load4(src, at + (upper ? e - half : e + half), DT, o);
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const float a = __fmul_rn(x[h][4 * (k & 1) + q], c[4 * k + q]), d = __fmul_rn(o[q], s[4 * k + q]);
                        x[h][4 * (k & 1) + q] = upper ? __fadd_rn(a, d) : __fsub_rn(a, d);
                    }
                }
            }
            __syncwarp();                        // queries may be turned in place
        }
    }
};

constexpr unsigned kRopeWarps = 4;               // a block

// (five blocks an SM: registers for four units in flight; seven blocks with spilled registers
// took 2% longer)
template <int DH, int MODE, int DT>
__global__ void __launch_bounds__(32 * kRopeWarps, MODE == 2 ? 4 : 5)
    rope_append_kernel(const __grid_constant__ RopeAppendParams p, int split)
{
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int LPR = DH / 16, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const unsigned w = blockIdx.x * kRopeWarps + (threadIdx.x >> 5);
    const unsigned token = w / (unsigned)split;
    if (token >= (unsigned)(p.rows.batch * p.n_new)) return;
    const int b = (int)(token / (unsigned)p.n_new), j = (int)(token - (unsigned)b * (unsigned)p.n_new);
    const int count = p.d_count ? min(p.d_count[b], p.n_new) : p.n_new;
    if (j >= count) return;
    const int first = p.d_pos[b];
    const int64_t pos = (int64_t)first + j;
    // the rope position of the sequence's token at index `at`, and whether the table has it
    auto rope_pos = [&](int64_t at) -> int64_t { return p.d_rope_pos ? p.d_rope_pos[(int64_t)b * p.n_new + at] : first + at; };
    auto in_table = [&](int64_t rp) { return rp >= 0 && rp < p.table_len; };
    const int64_t rp = rope_pos(j);
    if (!in_table(rp)) return;

    const int sub = lane / LPR, t = lane % LPR;
    Turn<DH, MODE> turn;
    turn.load(p.table + rp * (p.rot >> 1), p.rot, t);
    // A unit is RPW heads of a tensor; behind the last head a lane works on that one again, and
    // stores nothing.
    auto row_of = [&](const RowsView &r) { return b * r.batch_stride + j * r.token_stride; };
    const int Hq = p.q_in.data ? p.n_q_heads : 0, Hkv = p.rows.heads;
    const int nq = (Hq + RPW - 1) / RPW, nk = (Hkv + RPW - 1) / RPW;
    int i = (int)(w - token * (unsigned)split);
    if (i < nq) {
        constexpr int U = DT == KVQ_F32 || MODE == 2 ? 2 : 4;            // units in flight
        const int64_t from = row_of(p.q_in), to = row_of(p.q_out) + 8 * t;
#pragma unroll 1
        for (; i < nq; i += U * split) {
            Raw16<DT> raw[U];
#pragma unroll
            for (int u = 0; u < U; u++)
                if (u == 0 || i + u * split < nq)
                    raw[u].template load<DH>(p.q_in.data, from + min((i + u * split) * RPW + sub, Hq - 1) * DH + 8 * t);
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int head = (i + u * split) * RPW + sub;
                if (u > 0 && i + u * split >= nq) break;
                float x[2][8];
                raw[u].values(x);
                turn.template apply<DT>(x, p.q_in.data, from + min(head, Hq - 1) * DH);
                if (head < Hq) {
                    store8(p.q_out.data, to + head * DH, DT, x[0]);
                    store8(p.q_out.data, to + head * DH + DH / 2, DT, x[1]);
                }
            }
        }
        while (i - split >= nq) i -= split;      // (units past the last query's were skipped)
    }
    i -= nq;
    // a token that a later token of this call overwrites in the ring is not stored (one that is
    // skipped overwrites nothing)
    bool keep = true;
    if (p.rows.window > 0 && pos >= p.rows.n_anchor)
#pragma unroll 1
        for (int64_t at = (int64_t)j + p.rows.window; keep && at < count; at += p.rows.window) keep = !in_table(rope_pos(at));
    const int64_t row0 = keep ? cache_row(p.rows, b, 0, pos) : -1;       // head 0's row; heads lie apart by:
    const int64_t head_rows = p.rows.block_table ? kPageTokens : p.rows.cap;
    const int64_t from_k = row_of(p.k_in), from_v = row_of(p.v_in);
    auto load = [&](int at, Raw16<DT> &raw) {
        const bool is_v = at >= nk;
        const int head = min((is_v ? at - nk : at) * RPW + sub, Hkv - 1);
        raw.template load<DH>(is_v ? p.v_in.data : p.k_in.data, (is_v ? from_v : from_k) + head * DH + 8 * t);
    };
    Raw16<DT> raw, next;
    if (i < 2 * nk) load(i, next);
#pragma unroll 1
    for (; i < 2 * nk; i += split) {
        raw = next;
        if (i + split < 2 * nk) load(i + split, next);
        const bool is_v = i >= nk;
        const int head = (is_v ? i - nk : i) * RPW + sub;
        float x[2][8];
        raw.values(x);
        if (!is_v) turn.template apply<DT>(x, p.k_in.data, from_k + min(head, Hkv - 1) * DH);
        const int bits = is_v ? p.v.bits : p.k.bits, gshift = __ffs(is_v ? p.v.group : p.k.group) - 1;
        uint8_t *codes = is_v ? p.v.codes : p.k.codes;
        __half *scales = is_v ? p.v.scales : p.k.scales;
        const bool active = head < Hkv && row0 >= 0;
        const int64_t cr = active ? row0 + head * head_rows : 0;
        if (bits != 16 && p.fmt != KVQ_FMT_TENSOR) scales += cr * ((DH >> gshift) * scale_vals(p.fmt));
        quantize_row16<DH>(x, active, t, bits, gshift, p.fmt, codes + cr * (DH * bits / 8), scales);
    }
}

template <int DH, int MODE>
cudaError_t launch_append(const RopeAppendParams &p, unsigned blocks, int split, cudaStream_t stream)
{
    auto kernel = p.dtype == KVQ_F32   ? rope_append_kernel<DH, MODE, KVQ_F32>
                  : p.dtype == KVQ_F16 ? rope_append_kernel<DH, MODE, KVQ_F16>
                                       : rope_append_kernel<DH, MODE, KVQ_BF16>;
    return launch_dependent(kernel, blocks, 32 * kRopeWarps, 0, stream, p, split);
}

template <int DH>
cudaError_t launch_append_dh(const RopeAppendParams &p, unsigned blocks, int split, cudaStream_t stream)
{
    if (p.interleaved) return launch_append<DH, 1>(p, blocks, split, stream);
    if (p.rot == DH) return launch_append<DH, 0>(p, blocks, split, stream);
    return launch_append<DH, 2>(p, blocks, split, stream);
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
    const int rpw = 512 / p.dh;
    const int rows = ((p.q_in.data ? p.n_q_heads : 0) + rpw - 1) / rpw + 2 * ((p.rows.heads + rpw - 1) / rpw);
    // enough warps for 32 on every SM, as long as each keeps a row (with twice as many 2 x 4096
    // tokens took 1% longer, with four times as many 6%: (cos, sin) are read once a warp)
    int64_t split = (148 * 32 + tokens - 1) / tokens;
    if (split > rows) split = rows;
    if (split < 1) split = 1;
    const int64_t blocks = (tokens * split + kRopeWarps - 1) / kRopeWarps;
    if (blocks > 0x1fffffff) return cudaErrorInvalidValue;
    return p.dh == 128 ? launch_append_dh<128>(p, (unsigned)blocks, (int)split, stream)
                       : launch_append_dh<64>(p, (unsigned)blocks, (int)split, stream);
}

}  // namespace kvq
