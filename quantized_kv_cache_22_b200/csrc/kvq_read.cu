// kvq_read.cu -- cached rows back as 16- or 32-bit values, and the move of an accepted
// draft path's rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_internal.h"
#include "kvq_dequant.cuh"

namespace kvq {
namespace {

// A thread turns eight neighbouring elements of a row into values: 16 lanes a 128-element
// row, so that a warp's loads and stores are contiguous runs.  A block takes one head's
// kReadTokens consecutive tokens of K or of V: its code reads are one contiguous range.
constexpr int kReadThreads = 256;
constexpr int kReadUnroll = 4;

template <int BITS>
__device__ __forceinline__ void read_rows(const ReadParams &p, const CacheTensor &t, const RowsView &out, int b,
                                          int head, int j0, int count, int first)
{
    const int chunks = p.dim / 8;                        // 8-element chunks of a row
    const int per_pass = kReadThreads / min(chunks, kReadThreads);   // rows a pass handles
    const int lane_row = threadIdx.x / min(chunks, kReadThreads);
    if (lane_row >= per_pass) return;
    const int pairs = scale_vals(p.fmt);
    for (int ch = threadIdx.x % min(chunks, kReadThreads); ch < chunks; ch += kReadThreads) {
        int64_t row[kReadUnroll];
        Codes8<BITS> code[kReadUnroll];
        __half2 sc[kReadUnroll];
#pragma unroll
        for (int u = 0; u < kReadUnroll; u++) {
            const int j = j0 + u * per_pass + lane_row;
            row[u] = j < count ? cache_row(p.rows, b, head, (int64_t)first + j) : -1;
            if (row[u] < 0) continue;
            code[u].load(t.codes + row[u] * ((int64_t)p.dim * BITS / 8), ch);
            if constexpr (BITS != 16) {
                const __half *s = p.fmt == KVQ_FMT_TENSOR
                    ? t.scales : t.scales + (row[u] * (p.dim / t.group) + ch * 8 / t.group) * pairs;
                sc[u] = __halves2half2(s[0], p.fmt == KVQ_FMT_ASYM ? s[1] : __ushort_as_half(0));
            }
        }
#pragma unroll
        for (int u = 0; u < kReadUnroll; u++) {
            if (row[u] < 0) continue;
            const int j = j0 + u * per_pass + lane_row;
            float x[8];
            code[u].values(x, p.fmt);
            if constexpr (BITS != 16) {
                const float s = __low2float(sc[u]), z = __high2float(sc[u]);
#pragma unroll
                for (int e = 0; e < 8; e++) x[e] = (p.fmt == KVQ_FMT_ASYM ? x[e] - z : x[e]) * s;
            }
            store8(out.data, b * out.batch_stride + j * out.token_stride + (int64_t)head * p.dim + ch * 8,
                   p.out_dtype, x);
        }
    }
}

__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p, int tiles,
                                                            int tile_tokens)
{
    int64_t i = blockIdx.x;
    const int tile = (int)(i % tiles);
    i /= tiles;
    const int which = p.out[0].data == nullptr ? 1 : (p.out[1].data == nullptr ? 0 : (int)(i & 1));
    if (p.out[0].data != nullptr && p.out[1].data != nullptr) i >>= 1;
    const int head = (int)(i % p.rows.heads);
    const int b = (int)(i / p.rows.heads);
    const int count = p.d_count ? min(p.d_count[b], p.n) : p.n;
    const int j0 = tile * tile_tokens;
    if (j0 >= count) return;
    const int first = p.d_pos[b];
    const CacheTensor &t = p.t[which];
    if (t.bits == 8)
        read_rows<8>(p, t, p.out[which], b, head, j0, count, first);
    else if (t.bits == 4)
        read_rows<4>(p, t, p.out[which], b, head, j0, count, first);
    else
        read_rows<16>(p, t, p.out[which], b, head, j0, count, first);
}

// One warp moves the path's rows of one (layer, sequence, head) of K or of V.  The path is
// strictly ascending, so path[i] >= i: a source row of a batch is never the target of an
// earlier batch, and inside a batch every load comes before every store.
constexpr int kCommitBatch = 8;   // rows in flight

template <typename W>
__device__ __forceinline__ void move_rows(uint8_t *base, int64_t bytes, const CommitParams &p, const CacheRows &rows,
                                          int b, int head, int len, int path_lo, int path_hi, int m, int lane)
{
    const int words = (int)(bytes / (int64_t)sizeof(W));      // 1 .. 32 per row
    const int per = 32 / words;                               // rows the warp holds at a time
    const int sub = lane / words, col = lane % words;
    for (int i0 = 0; i0 < m; i0 += per * kCommitBatch) {
        W v[kCommitBatch];
        int64_t to[kCommitBatch];
#pragma unroll
        for (int u = 0; u < kCommitBatch; u++) {
            const int i = i0 + u * per + sub;
            const int lo = __shfl_sync(0xffffffffu, path_lo, i & 31), hi = __shfl_sync(0xffffffffu, path_hi, i & 31);
            const int from = i < 32 ? lo : hi;
            to[u] = -1;
            if (sub >= per || i >= m || from == i) continue;
            const int64_t src = cache_row(rows, b, head, (int64_t)len + from);
            const int64_t dst = cache_row(rows, b, head, (int64_t)len + i);
            if (src < 0 || dst < 0) continue;
            v[u] = reinterpret_cast<const W *>(base + src * bytes)[col];
            to[u] = dst;
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < kCommitBatch; u++)
            if (to[u] >= 0) reinterpret_cast<W *>(base + to[u] * bytes)[col] = v[u];
        __syncwarp();
    }
}

__device__ __forceinline__ void move_rows_any(uint8_t *base, int bytes, const CommitParams &p, const CacheRows &rows,
                                              int b, int head, int len, int lo, int hi, int m, int lane)
{
    if (bytes % 16 == 0)
        move_rows<uint4>(base, bytes, p, rows, b, head, len, lo, hi, m, lane);
    else if (bytes % 4 == 0)
        move_rows<uint32_t>(base, bytes, p, rows, b, head, len, lo, hi, m, lane);
    else
        move_rows<uint16_t>(base, bytes, p, rows, b, head, len, lo, hi, m, lane);
}

__global__ void __launch_bounds__(256) commit_kernel(const __grid_constant__ CommitParams p)
{
    const int lane = threadIdx.x & 31;
    int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t total = (int64_t)p.n_layers * p.rows.batch * p.rows.heads * 2;
    if (i >= total) return;
    const int which = (int)(i & 1);
    i >>= 1;
    const int head = (int)(i % p.rows.heads);
    i /= p.rows.heads;
    const int b = (int)(i % p.rows.batch);
    const int layer = (int)(i / p.rows.batch);
    int len = p.d_len[b];
    len = len < 0 ? 0 : (len > p.rows.cap ? p.rows.cap : len);

    // the path's valid prefix: strictly ascending indices below n_tree
    int m = p.d_n_path[b];
    m = m < 0 ? 0 : (m > p.path_stride ? p.path_stride : m);
    const int32_t *path = p.d_path + (int64_t)b * p.path_stride;
    const int lo = lane < m ? path[lane] : -1;
    const int hi = lane + 32 < m ? path[lane + 32] : -1;
    int before_lo = __shfl_up_sync(0xffffffffu, lo, 1), before_hi = __shfl_up_sync(0xffffffffu, hi, 1);
    const int last_lo = __shfl_sync(0xffffffffu, lo, 31);
    if (lane == 0) {
        before_lo = -1;
        before_hi = last_lo;
    }
    const unsigned ok_lo = __ballot_sync(0xffffffffu, lane < m && lo > before_lo && lo < p.n_tree);
    const unsigned ok_hi = __ballot_sync(0xffffffffu, lane + 32 < m && hi > before_hi && hi < p.n_tree);
    m = ~ok_lo ? __ffs(~ok_lo) - 1 : 32 + (~ok_hi ? __ffs(~ok_hi) - 1 : 32);

    if (which == 0 && head == 0 && layer == 0 && lane == 0 && p.d_len_out) p.d_len_out[b] = len + m;
    CacheRows rows = p.rows;
    rows.block_table = p.table[layer];
    move_rows_any(p.codes[which][layer], p.row_bytes[which], p, rows, b, head, len, lo, hi, m, lane);
    if (p.scale_bytes[which])
        move_rows_any(reinterpret_cast<uint8_t *>(p.scales[which][layer]), p.scale_bytes[which], p, rows, b, head,
                      len, lo, hi, m, lane);
}

}  // namespace

cudaError_t launch_read(const ReadParams &p, cudaStream_t stream)
{
    const int chunks = p.dim / 8 < kReadThreads ? p.dim / 8 : kReadThreads;
    const int tile_tokens = kReadThreads / chunks * kReadUnroll;
    const int tiles = (p.n + tile_tokens - 1) / tile_tokens;
    const int both = (p.out[0].data != nullptr) + (p.out[1].data != nullptr);
    const int64_t blocks = (int64_t)p.rows.batch * p.rows.heads * both * tiles;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    (void)cudaGetLastError();
    read_kernel<<<(unsigned)blocks, kReadThreads, 0, stream>>>(p, tiles, tile_tokens);
    return cudaGetLastError();
}

cudaError_t launch_commit(const CommitParams &p, cudaStream_t stream)
{
    const int64_t warps = (int64_t)p.n_layers * p.rows.batch * p.rows.heads * 2;
    const int64_t blocks = (warps + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    (void)cudaGetLastError();
    commit_kernel<<<(unsigned)blocks, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace kvq
