// kvq_read.cu -- cached rows back as 16- or 32-bit values, and the move of an accepted
// draft path's rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_internal.h"
#include "kvq_dequant.cuh"

namespace kvq {
namespace {

// Memory-bound: bytes of codes and scales in, bytes of values out, nothing reused.  A thread
// turns pieces of eight elements into values, sixteen (eight) lanes a row of 128 (64) elements,
// so that a warp's loads and stores are whole runs of a row; it takes kReadUnroll rows at a
// time, all their loads in flight first (one row a time left HBM at 2.7 TB/s).  A block takes
// consecutive tokens of one head of K or of V, whose codes are one contiguous range.
// Every code is exact in f16.  For F16 outputs the product with the scale is taken in f16:
// rounded once from the exact product, it is what fp32 (exact) and a rounding would give.
constexpr int kReadThreads = 256;
constexpr int kReadUnroll = 8;

template <int KIND>
__device__ __forceinline__ void read_rows(const ReadParams &p, const CacheTensor &t, const RowsView &out, int b,
                                          int head, int j0, int count, int first)
{
    const int chunks = p.dim / 8;                        // 8-element pieces of a row
    const int lanes = min(chunks, kReadThreads);
    const int per_pass = kReadThreads / lanes;           // rows a pass handles
    const int lane_row = threadIdx.x / lanes;
    if (lane_row >= per_pass) return;
    constexpr int PAIR = KIND == K_ASYM ? 2 : 1;
    const bool tensor = p.fmt == KVQ_FMT_TENSOR;
    const int ng = p.dim / t.group, gshift = t.group == 32 ? 5 : t.group == 64 ? 6 : 7;
    const int64_t row_bytes = (int64_t)chunks * Raw<KIND>::BYTES;
#pragma unroll 1
    for (int ch = threadIdx.x % lanes; ch < chunks; ch += lanes) {
        const int g = (ch * 8) >> gshift;
        bool live[kReadUnroll];
        Raw<KIND> raw[kReadUnroll];
        uint32_t sc[kReadUnroll];                        // scale, zero-point << 16
#pragma unroll
        for (int u = 0; u < kReadUnroll; u++) {
            const int j = j0 + u * per_pass + lane_row;
            const int64_t row = j < count ? cache_row(p.rows, b, head, (int64_t)first + j) : -1;
            live[u] = row >= 0;
            sc[u] = 0x3c00u;
            if (!live[u]) continue;
            raw[u].w = __ldcs(reinterpret_cast<const decltype(raw[u].w) *>(t.codes + row * row_bytes + ch * Raw<KIND>::BYTES));
            if constexpr (KIND != K_F16) {
                const uint16_t *s = reinterpret_cast<const uint16_t *>(t.scales) + (tensor ? 0 : (row * ng + g) * PAIR);
                sc[u] = KIND == K_ASYM ? *reinterpret_cast<const uint32_t *>(s) : *s;
            }
        }
#pragma unroll
        for (int u = 0; u < kReadUnroll; u++) {
            if (!live[u]) continue;
            const int j = j0 + u * per_pass + lane_row;
            uint32_t h[4];
            uint32_t zero = 0u;
            if constexpr (KIND == K_ASYM) zero = hadd2_u32((sc[u] >> 16) * 0x10001u, 0x64006400u);
            codes_f16<KIND>(raw[u], zero, h);
            const int64_t at = b * out.batch_stride + j * out.token_stride + (int64_t)head * p.dim + ch * 8;
            if (p.out_dtype == KVQ_F16) {
                if constexpr (KIND != K_F16) {
                    const uint32_t s2 = (sc[u] & 0xffffu) * 0x10001u;
#pragma unroll
                    for (int k = 0; k < 4; k++) h[k] = hmul2_u32(h[k], s2);
                }
                __stcs(reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out.data) + at), make_uint4(h[0], h[1], h[2], h[3]));
                continue;
            }
            const float s = KIND == K_F16 ? 1.f : __half2float(__ushort_as_half((unsigned short)sc[u]));
            float x[8];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const float2 v = unpack_half2(h[k]);
                x[2 * k] = v.x * s;
                x[2 * k + 1] = v.y * s;
            }
            store8(out.data, at, p.out_dtype, x);
        }
    }
}

__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p, int tiles,
                                                            int tile_tokens)
{
    grid_dependency_wait();
    grid_launch_dependents();
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
    switch (kind_of(t.bits, p.fmt)) {
    case K_INT8: return read_rows<K_INT8>(p, t, p.out[which], b, head, j0, count, first);
    case K_INT4: return read_rows<K_INT4>(p, t, p.out[which], b, head, j0, count, first);
    case K_E4M3: return read_rows<K_E4M3>(p, t, p.out[which], b, head, j0, count, first);
    case K_ASYM: return read_rows<K_ASYM>(p, t, p.out[which], b, head, j0, count, first);
    default: return read_rows<K_F16>(p, t, p.out[which], b, head, j0, count, first);
    }
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
    grid_dependency_wait();
    grid_launch_dependents();
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
    return launch_dependent(read_kernel, (unsigned)blocks, kReadThreads, 0, stream, p, tiles, tile_tokens);
}

cudaError_t launch_commit(const CommitParams &p, cudaStream_t stream)
{
    const int64_t warps = (int64_t)p.n_layers * p.rows.batch * p.rows.heads * 2;
    const int64_t blocks = (warps + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(commit_kernel, (unsigned)blocks, 256, 0, stream, p);
}

}  // namespace kvq
