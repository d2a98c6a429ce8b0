// kvq_tree.cu -- attention of a tree of drafted tokens over a quantised cache.
//
// One block takes eight query rows (a row: drafted token i, query head g of the KV head)
// of one (sequence, KV head); it walks the cache in tiles of 32 tokens that all threads
// dequantise into shared memory as fp32, and each warp keeps one row's running maximum,
// sum and output.
#include "kvq_internal.h"
#include "kvq_dequant.cuh"

namespace kvq {
namespace {

constexpr int kRows = 8, kTile = 32;

template <int BITS>
__device__ __forceinline__ void fill(float *dst, int stride, const TreeParams &p, const CacheTensor &t, int b, int head,
                                     int t0, int total)
{
    const int chunks = p.dh / 8;
    for (int i = threadIdx.x; i < kTile * chunks; i += blockDim.x) {
        const int tok = i / chunks, ch = i % chunks;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const int64_t row = t0 + tok < total ? cache_row(p.rows, b, head, t0 + tok) : -1;
        if (row >= 0) {
            Codes8<BITS> c;
            c.load(t.codes + row * ((int64_t)p.dh * BITS / 8), ch);
            c.values(x, p.fmt);
            if (BITS != 16) {
                const __half *s = p.fmt == KVQ_FMT_TENSOR
                    ? t.scales : t.scales + (row * (p.dh / t.group) + ch * 8 / t.group) * scale_vals(p.fmt);
                const float z = p.fmt == KVQ_FMT_ASYM ? __half2float(s[1]) : 0.f;
                for (int e = 0; e < 8; e++) x[e] = (x[e] - z) * __half2float(s[0]);
            }
        }
        for (int e = 0; e < 8; e++) dst[tok * stride + ch * 8 + e] = x[e];
    }
}

__device__ __forceinline__ void fill_any(float *dst, int stride, const TreeParams &p, const CacheTensor &t, int b,
                                         int head, int t0, int total)
{
    if (t.bits == 8) fill<8>(dst, stride, p, t, b, head, t0, total);
    else if (t.bits == 4) fill<4>(dst, stride, p, t, b, head, t0, total);
    else fill<16>(dst, stride, p, t, b, head, t0, total);
}

__device__ __forceinline__ float load1(const void *x, int64_t i, int dtype)
{
    if (dtype == KVQ_F32) return static_cast<const float *>(x)[i];
    if (dtype == KVQ_F16) return __half2float(static_cast<const __half *>(x)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(x)[i]);
}

__global__ void __launch_bounds__(kRows * 32) tree_kernel(const __grid_constant__ TreeParams p, int row_tiles)
{
    __shared__ float ks[kTile * 129], vs[kTile * 129], qs[kRows * 128];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rt = blockIdx.x % row_tiles;
    const int head = (blockIdx.x / row_tiles) % p.rows.heads;
    const int b = blockIdx.x / row_tiles / p.rows.heads;
    const int dh = p.dh, stride = dh + 1;
    const int r = rt * kRows + warp, i = r / p.G, g = r % p.G;
    const int len = max(0, min(p.d_len[b], p.rows.cap));
    const int n = p.d_n_tree ? max(0, min(p.d_n_tree[b], p.n_tree)) : p.n_tree;
    const int total = min(len + n, p.rows.cap);
    const bool live = r < p.n_tree * p.G && i < n;
    const int64_t at = (((int64_t)b * p.n_tree + i) * p.n_q_heads + (int64_t)head * p.G + g) * dh;
    const uint64_t mask = !live ? 0 : p.d_mask ? p.d_mask[(int64_t)b * p.n_tree + i] : ~0ull >> (63 - i);
    if (live)
        for (int d = lane; d < dh; d += 32) qs[warp * dh + d] = load1(p.q, at + d, p.q_dtype) * p.tau_log2e;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int t0 = 0; t0 < total; t0 += kTile) {
        __syncthreads();
        fill_any(ks, stride, p, p.k, b, head, t0, total);
        fill_any(vs, stride, p, p.v, b, head, t0, total);
        __syncthreads();
        const int t = t0 + lane;
        const bool seen = live && (t < len || (t < total && (mask >> (t - len) & 1)));
        float s = 0.f;
        for (int d = 0; d < dh; d++) s += qs[warp * dh + d] * ks[lane * stride + d];
        if (!seen) s = -INFINITY;
        float mx = s;
        for (int x = 16; x; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
        if (mx == -INFINITY) continue;
        const float up = fmaxf(m, mx), alpha = exp2f(m - up);
        m = up;
        const float e = seen ? exp2f(s - m) : 0.f;
        l = l * alpha + e;
        for (int k = 0; k < 4; k++) o[k] *= alpha;
        for (int tt = 0; tt < kTile; tt++) {
            const float w = __shfl_sync(~0u, e, tt);
            if (w == 0.f) continue;
            for (int k = 0; k < dh / 32; k++) o[k] += w * vs[tt * stride + k * 32 + lane];
        }
    }
    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(~0u, l, x);
    if (!live) return;
    for (int k = 0; k < dh / 32; k++) {
        const float y = l > 0.f ? o[k] / l : (l == 0.f ? 0.f : l);
        const int64_t x = at + k * 32 + lane;
        if (p.out_dtype == KVQ_F32) static_cast<float *>(p.out)[x] = y;
        else if (p.out_dtype == KVQ_F16) static_cast<__half *>(p.out)[x] = __float2half_rn(y);
        else static_cast<__nv_bfloat16 *>(p.out)[x] = __float2bfloat16_rn(y);
    }
}

}  // namespace

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream)
{
    const int row_tiles = (p.n_tree * p.G + kRows - 1) / kRows;
    const int64_t blocks = (int64_t)p.rows.batch * p.rows.heads * row_tiles;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    (void)cudaGetLastError();
    tree_kernel<<<(unsigned)blocks, kRows * 32, 0, stream>>>(p, row_tiles);
    return cudaGetLastError();
}

}  // namespace kvq
