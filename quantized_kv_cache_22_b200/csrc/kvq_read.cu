// kvq_read.cu -- cached rows back as 16- or 32-bit values, and the move of an accepted
// draft path's rows.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kvq_internal.h"
#include "kvq_dequant.cuh"

namespace kvq {
namespace {

// Memory-bound: bytes of codes and scales in, bytes of values out, nothing reused; what keeps it
// from that bound is instructions.  So a lane turns two pieces of eight elements, one of each
// half of a row (8 lanes a row of 128 elements, whose loads and stores are whole runs of it),
// of kReadUnroll rows at a time, all their loads in flight first, and in a cache that is
// neither paged nor a ring (FLAT) addresses advance by constants.  A block takes consecutive
// tokens of one head of K or of V.
// 16 x 8192 tokens of 8 heads of 128, INT8 to f16: 139 to 146 us, 5.5 to 5.8 TB/s, 85 to 89% of
// what a copy reaches (two rows in flight: 150; the addresses of a paged cache: 149 against 145
// in the same run; one piece a lane: 174, three quarters of the issue slots taken).
// Every code is exact in f16.  For F16 outputs the product with the scale is taken in f16:
// rounded once from the exact product, it is what fp32 (exact) and a rounding would give.
constexpr int kReadThreads = 128;
constexpr int kReadUnroll = 4;

// eight codes times their scale, as eight values at dst
template <int KIND, int DT>
__device__ __forceinline__ void put8(const Raw<KIND> &raw, uint32_t sc, uint8_t *dst)
{
    uint32_t h[4];
    uint32_t zero = 0u;
    if constexpr (KIND == K_ASYM) zero = hadd2_u32((sc >> 16) * 0x10001u, 0x64006400u);
    codes_f16<KIND>(raw, zero, h);
    if constexpr (DT == KVQ_F16) {
        if constexpr (KIND != K_F16) {
            const uint32_t s2 = prmt(sc, 0u, 0x1010);
#pragma unroll
            for (int k = 0; k < 4; k++) h[k] = hmul2_u32(h[k], s2);
        }
        __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(h[0], h[1], h[2], h[3]));
    } else {
        const float s = KIND == K_F16 ? 1.f : __half2float(__ushort_as_half((unsigned short)sc));
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float2 v = unpack_half2(h[k]);
            x[2 * k] = v.x * s;
            x[2 * k + 1] = v.y * s;
        }
        store8(dst, 0, DT, x);
    }
}

template <int KIND, int DT, bool FLAT>
__device__ __forceinline__ void read_rows(const ReadParams &p, const CacheTensor &t, const RowsView &out, int b,
                                          int head, int j0, int count, int first)
{
    constexpr int BYTES = Raw<KIND>::BYTES, OUT = DT == KVQ_F32 ? 4 : 2;
    const int half = p.dim / 16;                         // 8-element pieces of half a row
    const int lanes = min(half, kReadThreads);
    const int per_pass = kReadThreads / lanes;           // rows a pass handles
    const int lane_row = threadIdx.x / lanes;
    if (lane_row >= per_pass) return;
    const bool tensor = p.fmt == KVQ_FMT_TENSOR;
    const int gshift = __ffs(t.group) - 1, ng = p.dim >> gshift;
    const int64_t row_bytes = (int64_t)half * (2 * BYTES);
    const int j = j0 + lane_row;
    const int64_t row0 = ((int64_t)b * p.rows.heads + head) * p.rows.cap + first + j;    // FLAT
#pragma unroll 1
    for (int ch = threadIdx.x - lane_row * lanes; ch < half; ch += lanes) {
        const int g0 = (ch * 8) >> gshift, g1 = ((ch + half) * 8) >> gshift;
        bool live[kReadUnroll];
        Raw<KIND> raw[kReadUnroll][2];
        uint32_t sc[kReadUnroll][2];                     // scale, zero-point << 16
#pragma unroll
        for (int u = 0; u < kReadUnroll; u++) {
            const int ju = j + u * per_pass;
            int64_t row;
            if constexpr (FLAT) {
                live[u] = ju < count && (unsigned)first + (unsigned)ju < (unsigned)p.rows.cap;
                row = row0 + u * per_pass;
            } else {
                row = ju < count ? cache_row(p.rows, b, head, (int64_t)first + ju) : -1;
                live[u] = row >= 0;
            }
            if (!live[u]) continue;
            const uint8_t *src = t.codes + row * row_bytes + ch * BYTES;
            raw[u][0].w = __ldcs(reinterpret_cast<const decltype(raw[u][0].w) *>(src));
            raw[u][1].w = __ldcs(reinterpret_cast<const decltype(raw[u][0].w) *>(src + half * BYTES));
            if constexpr (KIND != K_F16) {
                using S = typename std::conditional<KIND == K_ASYM, uint32_t, uint16_t>::type;
                const S *s = reinterpret_cast<const S *>(t.scales) + (tensor ? 0 : row * ng);
                sc[u][0] = s[tensor ? 0 : g0];
                sc[u][1] = g1 == g0 || tensor ? sc[u][0] : s[g1];
            }
        }
        uint8_t *dst = static_cast<uint8_t *>(out.data) +
                       (b * out.batch_stride + j * out.token_stride + (int64_t)head * p.dim + ch * 8) * OUT;
#pragma unroll
        for (int u = 0; u < kReadUnroll; u++) {
            if (live[u]) {
                put8<KIND, DT>(raw[u][0], sc[u][0], dst);
                put8<KIND, DT>(raw[u][1], sc[u][1], dst + half * (8 * OUT));
            }
            dst += per_pass * out.token_stride * OUT;
        }
    }
}

template <int DT, bool FLAT>
__global__ void __launch_bounds__(kReadThreads, 8) read_kernel(const __grid_constant__ ReadParams p, int tiles,
                                                            int tile_tokens)
{
    grid_dependency_wait();
    grid_launch_dependents();
    unsigned i = blockIdx.x / (unsigned)tiles;
    const int j0 = (int)(blockIdx.x - i * (unsigned)tiles) * tile_tokens;
    int which = p.out[0].data == nullptr;
    if (p.out[0].data != nullptr && p.out[1].data != nullptr) {
        which = (int)(i & 1);
        i >>= 1;
    }
    const int b = (int)(i / (unsigned)p.rows.heads), head = (int)(i - (unsigned)b * (unsigned)p.rows.heads);
    const int count = p.d_count ? min(p.d_count[b], p.n) : p.n;
    if (j0 >= count) return;
    const int first = p.d_pos[b];
    const CacheTensor &t = p.t[which];
    switch (kind_of(t.bits, p.fmt)) {
    case K_INT8: return read_rows<K_INT8, DT, FLAT>(p, t, p.out[which], b, head, j0, count, first);
    case K_INT4: return read_rows<K_INT4, DT, FLAT>(p, t, p.out[which], b, head, j0, count, first);
    case K_E4M3: return read_rows<K_E4M3, DT, FLAT>(p, t, p.out[which], b, head, j0, count, first);
    case K_ASYM: return read_rows<K_ASYM, DT, FLAT>(p, t, p.out[which], b, head, j0, count, first);
    default: return read_rows<K_F16, DT, FLAT>(p, t, p.out[which], b, head, j0, count, first);
    }
}

template <bool FLAT>
cudaError_t launch_read_as(const ReadParams &p, unsigned blocks, int tiles, int tile_tokens, cudaStream_t stream)
{
    auto kernel = p.out_dtype == KVQ_F32   ? read_kernel<KVQ_F32, FLAT>
                  : p.out_dtype == KVQ_F16 ? read_kernel<KVQ_F16, FLAT>
                                           : read_kernel<KVQ_BF16, FLAT>;
    return launch_dependent(kernel, blocks, kReadThreads, 0, stream, p, tiles, tile_tokens);
}

// One warp moves the path's rows of one (layer, sequence, head) of K or of V.  The path is
// strictly ascending, so path[i] >= i: a source row of a batch is never the target of an
// earlier batch, and inside a batch every load comes before every store.  Latency bounds it (the
// length, the path, then rows): 3.0 us for one sequence and layer, 9.3 for 16 sequences of 8
// heads in 32 layers, 20 MB.
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
    const int lanes = p.dim / 16 < kReadThreads ? p.dim / 16 : kReadThreads;
    const int tile_tokens = kReadThreads / lanes * kReadUnroll;
    const int tiles = (p.n + tile_tokens - 1) / tile_tokens;
    const int both = (p.out[0].data != nullptr) + (p.out[1].data != nullptr);
    const int64_t blocks = (int64_t)p.rows.batch * p.rows.heads * both * tiles;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return p.rows.window == 0 && p.rows.block_table == nullptr
               ? launch_read_as<true>(p, (unsigned)blocks, tiles, tile_tokens, stream)
               : launch_read_as<false>(p, (unsigned)blocks, tiles, tile_tokens, stream);
}

cudaError_t launch_commit(const CommitParams &p, cudaStream_t stream)
{
    const int64_t warps = (int64_t)p.n_layers * p.rows.batch * p.rows.heads * 2;
    const int64_t blocks = (warps + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(commit_kernel, (unsigned)blocks, 256, 0, stream, p);
}

}  // namespace kvq
