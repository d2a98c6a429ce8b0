// kvq_tree.cu -- attention of a tree of drafted tokens over a quantised cache, on the
// 5th-generation tensor cores.
//
// For each (sequence, KV head) the rows of a problem are its query rows: drafted token i and
// query head g of the KV head, row i G + g; up to 128 of them form a row tile (one row per
// TMEM lane).  With k^_t = code * scale,
//   s = tau q . k^_t,  p = softmax(s) over the attended t,  out = sum_t p_t v^_t.
//
// Work.  Persistent CTAs; a unit is one 128-token tile of one (sequence, KV head, row tile).
// All units are split evenly over the CTAs, whatever the lengths; a run of units of the same
// row tile inside a CTA is a segment.  A segment that is the whole row tile writes the output,
// others leave (sum, max, l) partials that tree_merge_kernel joins.
//
// Per tile.
//   * A producer thread copies the raw codes and scales (contiguous in either layout: one bulk
//     copy each) into a ring whose entries hold one tile of K or of V.
//   * Eight converter warps turn codes into f16 operands in 128-byte-swizzled shared memory:
//     every code (INT8, INT4, e4m3, code minus zero-point) is exact in f16.  One scale per row
//     stays outside the product.  Scales per group go in as x = code * (scale / 2^e) in two
//     f16 parts, hi = rn(x) and lo = x - hi (both exact: at most 8 + 11 significant bits), 2^e
//     being the power of two of the row's largest scale; the product then takes both parts.
//   * S = Q K^T: tcgen05.mma kind::f16, M = 128 rows, N = 128 tokens; Q in TMEM (rows scaled by
//     a power of two, fp32 rows in two parts), K from shared memory, fp32 accumulators in TMEM.
//   * Softmax: a thread owns a row.  z = s * scale_k + log2(scale_v) in log2 units, so that
//     P = 2^(z - m) is the probability times the value scale, rounded to f16 (the only
//     rounding below fp32 in the path; m keeps P between the subnormals and 2^14), and
//     l += P / scale_v.  m moves only when P would pass 2^14: then O in TMEM is rescaled.
//   * O += P V: A = P in TMEM (over S's columns), B = V, MN-major.
//   * Few rows: with at most 64 (32) rows Q is laid into TMEM two (four) times, and each copy's
//     warps take one half (quarter) of the tile's tokens with zeros in the rest of their P, so
//     that all four warps share the exponentials; the copies' sums are joined at the end.
// Double-buffered S and P let the tensor cores run a tile ahead of the softmax.
//
// Every wait is bounded; a give-up records KVQ_ERR_TIMEOUT in the workspace's status word.
#include <algorithm>
#include <mutex>

#include "kvq_internal.h"
#include "kvq_dequant.cuh"
#include "kvq_ptx.cuh"

namespace kvq {
namespace {

constexpr int TT = 128;                 // tokens of a tile
constexpr int kSoftWarps = 4, kConvWarps = 8;
constexpr int kProducerWarp = 4, kMmaWarp = 5, kConvWarp0 = 6;
constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
constexpr int kConvThreads = 16 * kConvWarps;   // of K, and of V
constexpr int kMaxEntries = 12;
constexpr unsigned FULL = 0xffffffffu;

constexpr uint32_t COL_S = 0, COL_O = 256, COL_Q = 384, COL_QLO = 448;   // TMEM columns
constexpr uint32_t PANEL = TT * 128;    // 64 f16 of every token

// P in [0, 2^14]: m starts 6 to 7 below the first chunk's maximum and follows when 14 is passed
constexpr float kHead = 6.f, kMoveAt = 14.f;

struct Work {
    long long n, u0;                    // all units, first unit of this CTA
    long long pre;                      // units before sequence b
    int p, n_units, b;                  // CTAs with work, units of this CTA, sequence of u0
};
struct Ctl {
    uint64_t full[kMaxEntries], empty[kMaxEntries];
    uint64_t kfull[2], vfull[2], sfull[2], pfull[2], pvdone[2], par[4], qfull, soft, drain;
    Work w;
    uint32_t tmem;
    int abort;
    float2 ml[TT];
};
// Per-token numbers of a tile, four tiles deep: the converters run at most two tiles ahead of
// the softmax.
struct Par {
    float sk[4][TT], lv[4][TT], iv[4][TT];
};
constexpr int STAGE_LD = 33;            // floats per row of the epilogue's 32-column staging

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// The loop of a wait whose first try failed, out of line: the roles' hot code has to stay small.
__device__ __noinline__ bool wait_slow(uint64_t *bar, uint32_t parity, int *abort_flag, uint64_t limit)
{
    return mbar_wait_bounded(bar, parity, abort_flag, limit);
}

// ------------------------------------------------------------------ work split
struct Seq {
    int len, n, total, tiles, rtn;      // cached, drafted, attended tokens; tiles; row tiles
};
__device__ __forceinline__ Seq sequence(const TreeParams &p, int b)
{
    Seq s;
    s.len = max(0, min(p.d_len[b], p.rows.cap));
    s.n = p.d_n_tree ? max(0, min(p.d_n_tree[b], p.n_tree)) : p.n_tree;
    s.total = min(s.len + s.n, p.rows.cap);
    s.tiles = s.n > 0 ? (s.total + TT - 1) / TT : 0;
    s.rtn = (s.n * p.G + kTreeRows - 1) / kTreeRows;
    return s;
}

__device__ __forceinline__ long long range_begin(long long c, long long n, long long p) { return c * n / p; }
// the CTA whose range holds unit u
__device__ __forceinline__ int range_cta(long long u, long long n, long long p)
{
    return (int)(((u + 1) * p - 1) / n);
}

__device__ void find_work(const TreeParams &p, int lane, Work &w)
{
    const int Hkv = p.rows.heads, B = p.rows.batch;
    long long n = 0;
    for (int b = lane; b < B; b += 32) {
        const Seq s = sequence(p, b);
        n += (long long)s.tiles * s.rtn * Hkv;
    }
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(FULL, n, o);
    const long long P = n < gridDim.x ? n : gridDim.x;
    long long u0 = 0, u1 = 0;
    if (blockIdx.x < P) {
        u0 = range_begin(blockIdx.x, n, P);
        u1 = range_begin(blockIdx.x + 1, n, P);
    }
    int fb = 0;
    long long pre = 0, acc = 0;
    for (int b0 = 0; b0 < B && u1 > u0; b0 += 32) {
        const int b = b0 + lane;
        long long units = 0;
        if (b < B) {
            const Seq s = sequence(p, b);
            units = (long long)s.tiles * s.rtn * Hkv;
        }
        long long incl = units;
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += v;
        }
        const long long excl = acc + incl - units;
        const unsigned hit = __ballot_sync(FULL, excl <= u0 && u0 < excl + units);
        if (hit) {
            const int src = __ffs(hit) - 1;
            fb = __shfl_sync(FULL, b, src);
            pre = __shfl_sync(FULL, excl, src);
            break;
        }
        acc += __shfl_sync(FULL, incl, 31);
    }
    if (lane == 0) {
        w.n = n;
        w.u0 = u0;
        w.pre = pre;
        w.p = (int)P;
        w.n_units = (int)(u1 - u0);
        w.b = fb;
    }
}

// Walks the units of the CTA; every role keeps its own.
struct Walk {
    int b, inner, tile;                 // inner = KV head * row tiles + row tile
    Seq s;
    __device__ __forceinline__ void start(const TreeParams &p, const Work &w)
    {
        b = w.b;
        s = sequence(p, b);
        const int off = (int)(w.u0 - w.pre);
        inner = off / s.tiles;
        tile = off % s.tiles;
    }
    __device__ __forceinline__ void next(const TreeParams &p)
    {
        if (++tile < s.tiles) return;
        tile = 0;
        if (++inner < p.rows.heads * s.rtn) return;
        inner = 0;
        while (++b < p.rows.batch) {
            s = sequence(p, b);
            if (s.tiles) return;
        }
    }
};

// ------------------------------------------------------------------ codes to f16
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

// Scales of one token as the converters see them.
struct RowScale {
    int e;        // exponent of the largest group scale (grouped)
    bool bad;     // a scale or zero-point that is not a finite number
};
template <int KIND>
__device__ __forceinline__ RowScale row_scale(const uint16_t *sc, int t, int ng)
{
    constexpr int PAIR = KIND == K_ASYM ? 2 : 1;
    int m = 0, z = 0;
    for (int g = 0; g < ng; g++) {
        m = max(m, sc[(t * ng + g) * PAIR] & 0x7fff);
        if (KIND == K_ASYM) z = max(z, sc[(t * ng + g) * PAIR + 1] & 0x7fff);
    }
    RowScale r;
    r.bad = m >= 0x7c00 || z > 0x5bf8;              // 0x5bf8: 255
    r.e = m >= 0x400 ? (m >> 10) - 15 : -14;
    return r;
}

// One tile of K (ISV false) or V: raw codes and scales -> f16 operand rows, and the tile's
// per-token numbers: K the factor of a score; V log2 of the value scale and its inverse.
// Rows past nvalid of V are zeros (P is zero there, and stale bytes must not be NaN).
template <int DH, int KIND, bool GRP, bool ISV>
__device__ __forceinline__ void convert(const uint8_t *raw, const uint16_t *sc, uint8_t *dst, uint32_t lo_off,
                                        int nvalid, int ct, int ng, int gshift, float tensor, bool is_tensor,
                                        float *p0, float *p1)
{
    // A thread's pieces are eight codes wide: eight lanes a 64-element panel row (one
    // 128-byte operand row, so that their 16-byte stores hit all banks), four tokens a warp,
    // both panels of a 128-element row.  Neighbouring tokens take the panels in turns, so that
    // the lanes' loads hit all banks too.
    constexpr int ROW = DH / 8 * Raw<KIND>::BYTES, PANELS = DH / 64, RPP = kConvThreads / 8, PASSES = TT / RPP;
    constexpr int PAIR = KIND == K_ASYM ? 2 : 1;
    static_assert(kConvThreads == TT, "a thread a token");
    // elements that are not numbers: dropped, and the token's queries told by log2 = NaN
    constexpr bool CHECK = ISV && (KIND == K_E4M3 || KIND == K_F16);
    const int c = ct & 7, tr = ct >> 3, lane = ct & 31;
    const int turn = KIND == K_INT4 ? (tr >> 1) & 1 : tr & 1;

    auto params = [&](int t, bool bad) {
        if constexpr (GRP) {
            const RowScale r = row_scale<KIND>(sc, t, ng);
            if constexpr (ISV) {
                p0[t] = bad || r.bad ? __int_as_float(0x7fc00000) : (float)r.e;
                p1[t] = pow2i(-r.e);
            } else {
                p0[t] = pow2i(r.e);
            }
        } else {
            float s = 1.f;
            if (KIND != K_F16) s = is_tensor ? tensor : __half2float(__ushort_as_half(sc[t * PAIR]));
            if (KIND == K_ASYM) bad = bad || (sc[t * PAIR + 1] & 0x7fff) > 0x5bf8;
            if constexpr (ISV) {
                s = fabsf(s);
                if (!(s < INFINITY)) bad = true;
                // every value of the row is zero, or nothing may come of it (the inverse meets
                // P = 0 where the token is masked, so it has to be a number)
                if (s == 0.f || bad || t >= nvalid) s = 1.f;
                p0[t] = bad ? __int_as_float(0x7fc00000) : lg2(s);
                p1[t] = __frcp_rn(s);
            } else {
                p0[t] = s;
            }
        }
    };
    if (!CHECK) params(ct, false);                             // a thread a token

    const uint8_t *src = raw + tr * ROW + c * Raw<KIND>::BYTES;
    uint8_t *out = dst + tr * 128 + ((c ^ tr) & 7) * 16;      // (t ^ tr) & 7 = 0: RPP is a multiple of 8
    uint32_t bad_rows = 0;                                     // CHECK: bit u for pass u
    // (kept a loop: the roles' code together has to stay within the instruction cache)
#pragma unroll 1
    for (int pn = 0; pn < PANELS; pn++) {
        const int panel = PANELS == 2 ? pn ^ turn : 0;
        const int g = (c * 8 + 64 * panel) >> gshift;
        Raw<KIND> r[PASSES];
#pragma unroll
        for (int u = 0; u < PASSES; u++)
            r[u].w = *reinterpret_cast<const decltype(r[u].w) *>(src + u * RPP * ROW + panel * 8 * Raw<KIND>::BYTES);
#pragma unroll
        for (int u = 0; u < PASSES; u++) {
            const int t = u * RPP + tr;
            uint32_t h[4], zero = 0u;
            if constexpr (KIND == K_ASYM) {
                const uint32_t z = sc[(t * ng + g) * PAIR + 1];
                // a zero-point that is no number must not reach the rows that mask the token
                zero = hadd2_u32((ISV && z > 0x5bf8u ? 0u : z) * 0x10001u, 0x64006400u);
            }
            codes_f16<KIND>(r[u], zero, h);
            if constexpr (CHECK) {
                uint32_t any = 0;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t inf = ((h[k] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
                    any |= inf;
                    h[k] &= ~((inf >> 15) * 0xFFFFu);
                }
                const unsigned votes = __ballot_sync(FULL, any != 0);
                if ((votes >> (lane & 24)) & 0xFFu) bad_rows |= 1u << u;
            }
            uint8_t *d = out + u * RPP * 128 + panel * PANEL;
            if constexpr (GRP) {
                const RowScale rs = row_scale<KIND>(sc, t, ng);
                float s = __half2float(__ushort_as_half(sc[(t * ng + g) * PAIR])) * pow2i(-rs.e);
                if (ISV && rs.bad) s = 0.f;
                const uint32_t s2 = pack_half2(s, s);
                uint32_t l[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t hi = hmul2_u32(h[k], s2);
                    l[k] = hfma2_u32(h[k], s2, hi ^ 0x80008000u);
                    h[k] = hi;
                }
                *reinterpret_cast<uint4 *>(d + lo_off) = make_uint4(l[0], l[1], l[2], l[3]);
            }
            *reinterpret_cast<uint4 *>(d) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    if (CHECK && c == 0)
#pragma unroll 1
        for (int u = 0; u < PASSES; u++) params(u * RPP + tr, (bad_rows >> u) & 1u);
    if (ISV && nvalid < TT) {
        // the last tile: zeros past the sequence's end
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int u = 0; u < PASSES; u++) {
            if (u * RPP + tr < nvalid) continue;
            for (int pn = 0; pn < PANELS; pn++) {
                *reinterpret_cast<uint4 *>(out + u * RPP * 128 + pn * PANEL) = none;
                if (GRP) *reinterpret_cast<uint4 *>(out + u * RPP * 128 + pn * PANEL + lo_off) = none;
            }
        }
    }
}

template <int DH, bool ISV>
__device__ __forceinline__ void convert_any(const TreeParams &p, const uint8_t *entry, uint8_t *dst, int nvalid, int ct,
                                            float tensor, float *p0, float *p1)
{
    const CacheTensor &t = ISV ? p.v : p.k;
    const bool grp = ISV ? p.l.v_grouped : p.l.k_grouped;
    const int ng = DH / t.group, gshift = t.group == 32 ? 5 : t.group == 64 ? 6 : 7;
    const uint16_t *sc = reinterpret_cast<const uint16_t *>(entry + p.l.off_scales);
    const bool pt = p.fmt == KVQ_FMT_TENSOR;
#define KVQ_CONVERT(KIND)                                                                                          \
    if (grp)                                                                                                       \
        convert<DH, KIND, true, ISV>(entry, sc, dst, p.l.lo, nvalid, ct, ng, gshift, tensor, pt, p0, p1);            \
    else                                                                                                           \
        convert<DH, KIND, false, ISV>(entry, sc, dst, p.l.lo, nvalid, ct, ng, gshift, tensor, pt, p0, p1);
    switch (kind_of(t.bits, p.fmt)) {
    case K_INT8: KVQ_CONVERT(K_INT8) break;
    case K_INT4: KVQ_CONVERT(K_INT4) break;
    case K_E4M3: KVQ_CONVERT(K_E4M3) break;
    case K_ASYM: KVQ_CONVERT(K_ASYM) break;
    default:
        convert<DH, K_F16, false, ISV>(entry, sc, dst, p.l.lo, nvalid, ct, ng, gshift, tensor, pt, p0, p1);
        break;
    }
#undef KVQ_CONVERT
}

// ------------------------------------------------------------------ softmax
// 32 visible bits of tokens tok .. tok + 31 for a row whose drafted tokens are `mask`
__device__ __forceinline__ uint32_t visible(int tok, int len, uint64_t mask)
{
    const int d = tok - len;
    if (d <= -32) return FULL;
    if (d < 0) return ((1u << -d) - 1u) | (uint32_t)(mask << -d);
    return d < 64 ? (uint32_t)(mask >> d) : 0u;
}

// Two fp32 numbers in a register pair, and the packed instructions on them.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) { return (uint64_t)b << 32 | a; }
__device__ __forceinline__ uint64_t pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// z of 32 tokens (scores, fp32 accumulators in a, times the row's and the tokens' factors,
// plus log2 of the value scales; -inf where the row does not look), and their maximum
__device__ __forceinline__ float scores32(const uint32_t (&a)[32], const float *sk, const float *lv, float rf,
                                          uint32_t vis, uint64_t (&z)[16])
{
    const uint64_t rf2 = pair(rf, rf);
#pragma unroll
    for (int t = 0; t < 16; t += 2) {
        const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(sk + 2 * t);
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(lv + 2 * t);
        z[t] = fma2(mul2(pair(a[2 * t], a[2 * t + 1]), k.x), rf2, v.x);
        z[t + 1] = fma2(mul2(pair(a[2 * t + 2], a[2 * t + 3]), k.y), rf2, v.y);
    }
    if (vis != FULL) {
#pragma unroll
        for (int t = 0; t < 16; t++)
            z[t] = pair((vis >> (2 * t)) & 1u ? first(z[t]) : -INFINITY,
                        (vis >> (2 * t + 1)) & 1u ? second(z[t]) : -INFINITY);
    }
    float m0 = fmaxf(first(z[0]), second(z[0])), m1 = fmaxf(first(z[1]), second(z[1]));
#pragma unroll
    for (int t = 2; t < 16; t += 2) {
        m0 = fmaxf(m0, fmaxf(first(z[t]), second(z[t])));
        m1 = fmaxf(m1, fmaxf(first(z[t + 1]), second(z[t + 1])));
    }
    return fmaxf(m0, m1);
}

// P = 2^(z - m) of 32 tokens, rounded to f16, into 16 packed columns; returns their share of l
__device__ __forceinline__ float probs32(const uint64_t (&z)[16], const float *iv, float m, uint32_t (&w)[16])
{
    const uint64_t nm = pair(-m, -m);
    uint64_t l0 = 0, l1 = 0;
#pragma unroll
    for (int t = 0; t < 16; t += 2) {
        const ulonglong2 i = *reinterpret_cast<const ulonglong2 *>(iv + 2 * t);
        const uint64_t x = add2(z[t], nm), y = add2(z[t + 1], nm);
        const float a = ex2(first(x)), b = ex2(second(x)), c = ex2(first(y)), d = ex2(second(y));
        l0 = fma2(pair(a, b), i.x, l0);
        l1 = fma2(pair(c, d), i.y, l1);
        w[t] = pack_half2(a, b);
        w[t + 1] = pack_half2(c, d);
    }
    return (first(l0) + second(l0)) + (first(l1) + second(l1));
}

// ------------------------------------------------------------------ the kernel
template <int DH>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p)
{
    constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(TT >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t IDESC_O = (1u << 4) | (1u << 16) | ((uint32_t)(DH >> 3) << 17) | ((128u >> 4) << 24);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + p.l.off_ctl);
    Par *par = reinterpret_cast<Par *>(smem + p.l.off_par);
    int *abort_flag = &ctl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = p.l.entries, KB = p.l.k_bufs, VB = p.l.v_bufs;
    const uint64_t limit = p.timeout_ns;
    auto give_up = [&]() {
        *static_cast<volatile int *>(abort_flag) = 1;
        atomicExch(p.status, KVQ_ERR_TIMEOUT);
    };
    auto wait1 = [&](uint64_t *bar, int parity) {
        return mbar_try_wait(bar, parity & 1) || wait_slow(bar, parity & 1, abort_flag, limit);
    };
    // a wait of a whole warp: its lanes go on, or give up, together
    auto wait = [&](uint64_t *bar, int parity) {
        return __all_sync(FULL, wait1(bar, parity)) != 0;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < E; s++) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], kConvWarps / 2);
        }
        for (int j = 0; j < 2; j++) {
            mbar_init(&ctl->kfull[j], kConvWarps / 2);
            mbar_init(&ctl->vfull[j], kConvWarps / 2);
            mbar_init(&ctl->sfull[j], 1);
            mbar_init(&ctl->pfull[j], kSoftWarps);
            mbar_init(&ctl->pvdone[j], 1);
        }
        for (int j = 0; j < 4; j++) mbar_init(&ctl->par[j], kConvWarps);
        mbar_init(&ctl->qfull, kSoftWarps);
        mbar_init(&ctl->soft, kSoftWarps);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) find_work(p, lane, ctl->w);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Work w = ctl->w;
    const uint32_t tmem = ctl->tmem;
    const int n_units = w.n_units;

    if (warp == kProducerWarp) {
        // ====================== producer ======================
        if (lane == 0 && n_units > 0) {
            const uint64_t pol = l2_evict_first_policy();
            const int kr = DH * p.k.bits / 8, vr = DH * p.v.bits / 8;
            const bool ks = p.k.bits != 16 && p.fmt != KVQ_FMT_TENSOR, vs = p.v.bits != 16 && p.fmt != KVQ_FMT_TENSOR;
            const int ksb = DH / p.k.group * scale_vals(p.fmt) * 2, vsb = DH / p.v.group * scale_vals(p.fmt) * 2;
            Walk it;
            it.start(p, w);
            int e = 0, s = 0, use = 0;          // entries filled; the next one's place and use
            for (int i = 0; i < n_units; i++) {
                const int head = it.inner / it.s.rtn, t0 = it.tile * TT;
                const int nv = min(TT, it.s.total - t0);
                int64_t row;
                if (p.rows.block_table != nullptr) {
                    int page = p.rows.block_table[(int64_t)it.b * p.rows.max_pages + it.tile];
                    page = min(max(page, 0), p.rows.n_pages - 1);   // stay inside the pool
                    row = ((int64_t)page * p.rows.heads + head) * kPageTokens;
                } else {
                    row = ((int64_t)it.b * p.rows.heads + head) * p.rows.cap + t0;
                }
                const int nsc = (nv + 7) & ~7;      // rows whose scales are whole 16-byte pieces
                bool ok = true;
#pragma unroll 1
                for (int kv = 0; kv < 2; kv++, e++) {
                    if (use > 0 && !wait1(&ctl->empty[s], use - 1)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    const CacheTensor &t = kv ? p.v : p.k;
                    const int rb = kv ? vr : kr, sb = kv ? vsb : ksb;
                    const bool sc = kv ? vs : ks;
                    uint8_t *dst = smem + (uint32_t)s * p.l.entry_bytes;
                    mbar_arrive_expect_tx(&ctl->full[s], (uint32_t)(nv * rb + (sc ? nsc * sb : 0)));
                    bulk_load_hint(dst, t.codes + row * rb, (uint32_t)(nv * rb), &ctl->full[s], pol);
                    if (sc)
                        bulk_load_hint(dst + p.l.off_scales, reinterpret_cast<const uint8_t *>(t.scales) + row * sb,
                                       (uint32_t)(nsc * sb), &ctl->full[s], pol);
                    if (++s == E) {
                        s = 0;
                        ++use;
                    }
                }
                if (!ok) break;
                it.next(p);
            }
            // copies in flight land before the CTA ends, whatever the other roles did
            for (int k = e > E ? e - E : 0; k < e; k++) (void)mbar_wait_drain(&ctl->full[k % E], (k / E) & 1, limit);
        }
    } else if (warp == kMmaWarp) {
        // ====================== MMA issuer ======================
        if (lane == 0 && n_units > 0) {
            const uint32_t sbase = smem_u32(smem);
            const bool q2 = p.q_dtype == KVQ_F32;
            Walk it;
            it.start(p, w);
            int seg = -1;
            bool ok = true, first_prev = false;
            auto issue_pv = [&](int i, bool first) -> bool {
                const int j = i & 1, vb = i & (VB - 1);
                if (!wait1(&ctl->vfull[vb], i >> (VB - 1))) return false;
                if (!wait1(&ctl->pfull[j], i >> 1)) return false;
                tc_fence_after();
                const uint32_t v0 = sbase + p.l.off_v + (uint32_t)vb * p.l.v_bytes;
#pragma unroll 1
                for (int part = 0; part <= p.l.v_grouped; part++)
#pragma unroll
                    for (int kk = 0; kk < TT / 16; kk++)
                        umma_f16_ts(tmem + COL_O, tmem + COL_S + 128u * j + 8u * kk,
                                    sw128_mn_desc(v0 + part * p.l.lo + 2048u * kk, PANEL, 1024u), IDESC_O,
                                    first && part == 0 && kk == 0 ? 0u : 1u);
                umma_commit(&ctl->pvdone[j]);
                return true;
            };
            auto issue_s = [&](int i) -> bool {
                const int kb = i & (KB - 1);
                if (!wait1(&ctl->kfull[kb], i >> (KB - 1))) return false;
                tc_fence_after();
                const uint32_t k0 = sbase + p.l.off_k + (uint32_t)kb * p.l.k_bytes;
#pragma unroll 1
                for (int part = 0; part <= p.l.k_grouped; part++)
#pragma unroll 1
                    for (int qp = 0; qp <= (q2 ? 1 : 0); qp++)
#pragma unroll
                        for (int kk = 0; kk < DH / 16; kk++)
                            umma_f16_ts(tmem + COL_S + 128u * (i & 1), tmem + (qp ? COL_QLO : COL_Q) + 8u * kk,
                                        sw128_desc(k0 + part * p.l.lo + (uint32_t)(kk >> 2) * PANEL + 32u * (kk & 3)),
                                        IDESC_S, part == 0 && qp == 0 && kk == 0 ? 0u : 1u);
                umma_commit(&ctl->sfull[i & 1]);
                return true;
            };
            bool issued = false;
            for (int i = 0; i <= n_units && ok; i++) {
                const bool have = i < n_units;
                const bool first = have && (i == 0 || it.tile == 0);
                // a new segment's queries replace the old ones: its scores wait for the last P V
                if (i > 0 && (first || !have)) ok = issue_pv(i - 1, first_prev);
                if (ok && first) ok = wait1(&ctl->qfull, ++seg);
                if (ok && have) {
                    ok = issue_s(i);
                    issued |= ok;
                }
                if (ok && i > 0 && have && !first) ok = issue_pv(i - 1, first_prev);
                first_prev = first;
                if (have) it.next(p);
            }
            if (!ok) give_up();
            if (issued) {
                umma_commit(&ctl->drain);
                (void)mbar_wait_drain(&ctl->drain, 0, limit);
            }
        }
    } else if (warp >= kConvWarp0) {
        // ====================== converters ======================
        // four warps turn K tiles, four V tiles
        const int kv = warp >= kConvWarp0 + kConvWarps / 2;
        const int ct = (threadIdx.x - 32 * kConvWarp0) & (kConvThreads - 1);
        const CacheTensor &t = kv ? p.v : p.k;
        const float tensor = p.fmt == KVQ_FMT_TENSOR ? __half2float(t.scales[0]) : 1.f;
        const int bufs = kv ? VB : KB;
        uint8_t *tiles = smem + (kv ? p.l.off_v : p.l.off_k);
        const uint32_t tile_bytes = kv ? p.l.v_bytes : p.l.k_bytes;
        uint64_t *ready = kv ? ctl->vfull : ctl->kfull, *used = kv ? ctl->pvdone : ctl->sfull;
        Walk it;
        if (n_units > 0) it.start(p, w);
        bool ok = true;
        int s = kv, use = 0;
        for (int i = 0; i < n_units; i++) {
            const int nv = min(TT, it.s.total - it.tile * TT);
            ok = wait(&ctl->full[s], use);
            // the operand's last use: S, or P V, of tile i - bufs
            if (ok && i >= bufs) ok = wait(&used[(i - bufs) & 1], (i - bufs) >> 1);
            if (!ok) break;
            const uint8_t *entry = smem + (uint32_t)s * p.l.entry_bytes;
            const int buf = i & (bufs - 1);
            if (kv)
                convert_any<DH, true>(p, entry, tiles + (uint32_t)buf * tile_bytes, nv, ct, tensor, par->lv[i & 3],
                                      par->iv[i & 3]);
            else
                convert_any<DH, false>(p, entry, tiles + (uint32_t)buf * tile_bytes, nv, ct, tensor, par->sk[i & 3],
                                       nullptr);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&ctl->par[i & 3]);       // before the tile can be used, so that its
                mbar_arrive(&ready[buf]);            // phase is over when the slot comes round
                mbar_arrive(&ctl->empty[s]);
            }
            s += 2;
            if (s >= E) {
                s -= E;
                ++use;
            }
            it.next(p);
        }
        if (!ok) give_up();
    } else {
        // ====================== softmax ======================
        const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
        const int place = 32 * warp + lane;          // TMEM lane
        float *stage = reinterpret_cast<float *>(smem + p.l.off_stage);
        const float osign = p.fmt == KVQ_FMT_TENSOR && __half2float(p.v.scales[0]) < 0.f ? -1.f : 1.f;
        Walk it;
        if (n_units > 0) it.start(p, w);
        bool ok = true;
        int syncs = 0;
        auto soft_sync = [&]() {                     // the four warps meet
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->soft);
            const bool r = wait(&ctl->soft, syncs & 1);
            ++syncs;
            return r;
        };
        // What a thread keeps of its row; the next segment's is made while the last tile of the
        // current one is with the tensor cores.
        struct Row {
            int rows, copies, tb;                    // rows of the tile, their copies; first token of this copy
            float rf;                                // factor of a score: tau log2(e), the query's power of two
            uint64_t mask;                           // drafted tokens that the row attends
        };
        // this thread's row of the walk's segment, its query into TMEM
        auto open = [&](const Walk &o) {
            const int head = o.inner / o.s.rtn, rt = o.inner % o.s.rtn;
            Row x;
            x.rows = min(kTreeRows, o.s.n * p.G - rt * kTreeRows);
            x.copies = x.rows <= 32 ? 4 : x.rows <= 64 ? 2 : 1;
            const int r = place & (TT / x.copies - 1);
            x.tb = place - r;
            const int rr = rt * kTreeRows + r, qi = rr / p.G;
            const bool live = r < x.rows;
            const int64_t at = (((int64_t)o.b * p.n_tree + qi) * p.n_q_heads + (int64_t)head * p.G + rr % p.G) * DH;
            x.rf = p.tau_log2e;
            x.mask = 0;
            if (live) {
                const int nd = o.s.total - o.s.len;                  // drafted tokens that exist
                x.mask = p.d_mask ? p.d_mask[(int64_t)o.b * p.n_tree + qi] : ~0ull >> (63 - qi);
                x.mask &= nd > 0 ? ~0ull >> (64 - nd) : 0ull;
            }
            // bring the largest element of a row to [2^8, 2^9): f16 then holds bf16 elements, and
            // the first part of fp32 ones, as they are
            auto level = [&](float a) {
                if (!(a > 0.f && a < INFINITY)) return 1.f;
                const int ex = max((__float_as_int(a) >> 23) - 127, -110) - 8;
                x.rf = p.tau_log2e * pow2i(ex);
                return pow2i(-ex);
            };
            if (p.q_dtype != KVQ_F32) {
                uint4 u[DH / 8];
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at);
#pragma unroll
                for (int k = 0; k < DH / 8; k++) u[k] = live ? src[k] : make_uint4(0u, 0u, 0u, 0u);
                uint32_t *h = reinterpret_cast<uint32_t *>(u);
                if (p.q_dtype == KVQ_BF16) {
                    float a = 0.f;
#pragma unroll
                    for (int k = 0; k < DH / 2; k++)
                        a = fmaxf(a, fmaxf(fabsf(__uint_as_float(h[k] << 16)), fabsf(__uint_as_float(h[k] & 0xffff0000u))));
                    const float pre = level(a);
#pragma unroll
                    for (int k = 0; k < DH / 2; k++)
                        h[k] = pack_half2(__uint_as_float(h[k] << 16) * pre, __uint_as_float(h[k] & 0xffff0000u) * pre);
                }
#pragma unroll
                for (int k = 0; k < DH / 32; k++)
                    tmem_st16(tmem + COL_Q + lane_off + 16u * k, *reinterpret_cast<uint32_t(*)[16]>(h + 16 * k));
            } else {
                const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at);
                const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
                float a = 0.f;
#pragma unroll 4
                for (int k = 0; k < DH / 4; k++) {
                    const float4 f = live ? src[k] : none;
                    a = fmaxf(fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
                }
                const float pre = level(a);
#pragma unroll 1
                for (int c = 0; c < DH / 32; c++) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int k = 0; k < 8; k++) {
                        float4 f = live ? src[8 * c + k] : none;
                        f.x *= pre; f.y *= pre; f.z *= pre; f.w *= pre;
                        hi[2 * k] = pack_half2(f.x, f.y);
                        hi[2 * k + 1] = pack_half2(f.z, f.w);
                        const float2 b0 = unpack_half2(hi[2 * k]), b1 = unpack_half2(hi[2 * k + 1]);
                        lo[2 * k] = pack_half2(f.x - b0.x, f.y - b0.y);
                        lo[2 * k + 1] = pack_half2(f.z - b1.x, f.w - b1.y);
                    }
                    tmem_st16(tmem + COL_Q + lane_off + 16u * c, hi);
                    tmem_st16(tmem + COL_QLO + lane_off + 16u * c, lo);
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->qfull);
            return x;
        };
        float m = -INFINITY, l = 0.f;
        int seg0 = 0;                                // the segment's first unit in this CTA
        Row row{}, next{};
        if (n_units > 0) row = open(it);
        for (int i = 0; i < n_units; i++) {
            const int j = i & 1, t0 = it.tile * TT;
            const int copies = row.copies, tb = row.tb;
            const bool last = i == n_units - 1 || it.tile == it.s.tiles - 1;
            Walk ahead = it;
            ahead.next(p);

            // ---- scores of the tile
            ok = wait(&ctl->par[i & 3], i >> 2) &&
                 wait(&ctl->sfull[j], i >> 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_at = tmem + COL_S + 128u * j + lane_off;
            const float *sk = par->sk[i & 3] + tb, *lv = par->lv[i & 3] + tb, *iv = par->iv[i & 3] + tb;
            const bool whole = t0 + TT <= it.s.len;
            // one 32-token chunk at a time: its z, its maximum, its P over S's columns
            const int chunks = 4 / copies;
            const uint32_t p_at = s_at + (uint32_t)tb / 2;
#pragma unroll 1
            for (int c = 0; c < chunks; c++) {
                uint32_t a[32], pw[16];
                uint64_t z[16];
                tmem_ld32(s_at + tb + 32u * c, a);
                const uint32_t vis = whole ? FULL : visible(t0 + tb + 32 * c, it.s.len, row.mask);
                const float mx = scores32(a, sk + 32 * c, lv + 32 * c, row.rf, vis, z);
                const bool set = m == -INFINITY && mx > -INFINITY, up = !set && mx > m + kMoveAt;
                float alpha = 1.f;
                if (set || up) {
                    const float to = floorf(mx) - kHead;
                    if (up) alpha = ex2(m - to);             // m and to are whole: a power of two
                    m = to;
                    l *= alpha;
                }
                if (__any_sync(FULL, up)) {
                    // m moved too far for some row: O follows (every P V before this tile is in
                    // it; in a segment's first tile there is nothing yet), and this tile's P
                    if (i > seg0) {
                        if (!(ok = wait(&ctl->pvdone[j ^ 1], (i - 1) >> 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < DH / 32; x++) {
                            tmem_ld32(tmem + COL_O + lane_off + 32u * x, a);
#pragma unroll
                            for (int y = 0; y < 32; y++) a[y] = __float_as_uint(__uint_as_float(a[y]) * alpha);
                            tmem_st32(tmem + COL_O + lane_off + 32u * x, a);
                        }
                    }
                    const uint32_t alpha2 = pack_half2(alpha, alpha);
#pragma unroll 1
                    for (int x = 0; x < c; x++) {
                        tmem_st_wait();
                        tmem_ld16(p_at + 16u * x, pw);
#pragma unroll
                        for (int y = 0; y < 16; y++) pw[y] = hmul2_u32(pw[y], alpha2);
                        tmem_st16(p_at + 16u * x, pw);
                    }
                }
                l += probs32(z, iv + 32 * c, m == -INFINITY ? 0.f : m, pw);
                tmem_st16(p_at + 16u * c, pw);
            }
            if (!ok) break;
            if (copies > 1) {
                // the other copies' tokens
                uint32_t none[16];
#pragma unroll
                for (int x = 0; x < 16; x++) none[x] = 0u;
#pragma unroll 1
                for (int c = chunks; c < 4; c++) tmem_st16(s_at + (((uint32_t)tb / 2 + 16u * c) & 63u), none);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->pfull[j]);
            // every score of the segment is done: the next one's queries may come in
            if (last && i + 1 < n_units) next = open(ahead);

            // ---- the segment's last tile: join the copies, write the output or a partial
            if (last) {
                const int head = it.inner / it.s.rtn, rt = it.inner % it.s.rtn;
                const int nr = TT / copies, r = place - tb, rows = row.rows;
                float M = m, L = l;
                if (copies > 1) {
                    ctl->ml[place] = make_float2(m, l);
                    if (!(ok = soft_sync())) break;
                    M = -INFINITY;
                    L = 0.f;
                    for (int c = 0; c < copies; c++) M = fmaxf(M, ctl->ml[c * nr + r].x);
                    for (int c = 0; c < copies; c++) {
                        const float2 x = ctl->ml[c * nr + r];
                        L += x.x == -INFINITY ? 0.f : x.y * ex2(x.x - M);
                    }
                }
                float f = m == -INFINITY ? 0.f : ex2(m - M) * osign;
                const long long u0 = w.u0 + i - it.tile;
                const int ca = range_cta(u0, w.n, w.p), cb = range_cta(u0 + it.s.tiles - 1, w.n, w.p);
                const bool direct = ca == cb;
                // a CTA leaves two partials at most: of its first segment, and of its last
                const int slot = 2 * (int)blockIdx.x + (i - it.tile <= 0 ? 0 : 1);
                float *part = p.slots + (int64_t)slot * tree_slot_floats(p.slot_rows, DH);
                if (direct) f = L != 0.f ? f / L : 0.f;
                if (place == 0 && ca == (int)blockIdx.x)
                    p.seg[((int64_t)it.b * p.rows.heads + head) * p.row_tiles + rt] = make_int4(slot, ca, cb - ca + 1, 0);
                if (!direct && place < rows)
                    *reinterpret_cast<float2 *>(part + (int64_t)p.slot_rows * DH + 2 * place) = make_float2(M, L);
                // columns col .. col + 3 of a row of the tile
                auto put = [&](int rr, int col, const float (&y)[4]) {
                    if (!direct) {
                        *reinterpret_cast<float4 *>(part + (int64_t)rr * DH + col) = make_float4(y[0], y[1], y[2], y[3]);
                        return;
                    }
                    rr += rt * kTreeRows;
                    store4(p.out, (((int64_t)it.b * p.n_tree + rr / p.G) * p.n_q_heads + (int64_t)head * p.G + rr % p.G) * DH + col,
                           p.out_dtype, y);
                };
                if (!(ok = wait(&ctl->pvdone[j], i >> 1))) break;
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < DH / 32; c++) {
                    uint32_t o[32];
                    tmem_ld32(tmem + COL_O + lane_off + 32u * c, o);
                    if (copies == 1) {
                        if (place < rows)
#pragma unroll
                            for (int x = 0; x < 32; x += 4) {
                                float y[4];
#pragma unroll
                                for (int d = 0; d < 4; d++) y[d] = f == 0.f ? 0.f : __uint_as_float(o[x + d]) * f;
                                put(place, 32 * c + x, y);
                            }
                        continue;
                    }
                    if (c > 0 && !(ok = soft_sync())) break;         // the staging was read
#pragma unroll
                    for (int x = 0; x < 32; x++) stage[place * STAGE_LD + x] = f == 0.f ? 0.f : __uint_as_float(o[x]) * f;
                    if (!(ok = soft_sync())) break;
#pragma unroll 1
                    for (int x = place; x < rows * 8; x += TT) {
                        const int rr = x >> 3, col = (x & 7) * 4;
                        float y[4] = {0.f, 0.f, 0.f, 0.f};
                        for (int k = 0; k < copies; k++)
#pragma unroll
                            for (int d = 0; d < 4; d++) y[d] += stage[(k * nr + rr) * STAGE_LD + col + d];
                        put(rr, 32 * c + col, y);
                    }
                }
                if (!ok) break;
                row = next;
                m = -INFINITY;
                l = 0.f;
                seg0 = i + 1;
            }
            it = ahead;
        }
        if (!ok) give_up();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// One warp joins the partials of one row whose row tile several CTAs shared.
template <int DH>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int R = p.n_tree * p.G;
    if (i >= (int64_t)p.rows.batch * p.rows.heads * R) return;
    const int rr = (int)(i % R);
    const int head = (int)(i / R % p.rows.heads), b = (int)(i / R / p.rows.heads);
    const Seq s = sequence(p, b);
    if (rr >= s.n * p.G) return;
    const int4 seg = p.seg[((int64_t)b * p.rows.heads + head) * p.row_tiles + rr / kTreeRows];
    if (seg.z <= 1) return;
    const int r = rr % kTreeRows;
    const int64_t floats = tree_slot_floats(p.slot_rows, DH);
    auto slot = [&](int k) { return p.slots + (int64_t)(k == 0 ? seg.x : 2 * (seg.y + k)) * floats; };
    float M = -INFINITY;
    for (int k = lane; k < seg.z; k += 32) M = fmaxf(M, slot(k)[(int64_t)p.slot_rows * DH + 2 * r]);
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    constexpr int PER = DH / 32;
    float L = 0.f, y[PER];
#pragma unroll
    for (int d = 0; d < PER; d++) y[d] = 0.f;
#pragma unroll 4
    for (int k = 0; k < seg.z; k++) {
        const float *x = slot(k);
        const float2 ml = *reinterpret_cast<const float2 *>(x + (int64_t)p.slot_rows * DH + 2 * r);
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
        L = fmaf(ml.y, f, L);
#pragma unroll
        for (int d = 0; d < PER; d++) y[d] = fmaf(x[(int64_t)r * DH + lane * PER + d], f, y[d]);
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int64_t at = (((int64_t)b * p.n_tree + rr / p.G) * p.n_q_heads + (int64_t)head * p.G + rr % p.G) * DH + lane * PER;
#pragma unroll
    for (int d = 0; d < PER; d++) y[d] *= inv;
    if constexpr (PER == 4)
        store4(p.out, at, p.out_dtype, y);
    else
        store2(p.out, at, p.out_dtype, y);
}

uint32_t align_up(uint32_t x, uint32_t a) { return (x + a - 1) / a * a; }

template <int DH>
cudaError_t launch(const TreeParams &p, cudaStream_t stream)
{
    void *fn = reinterpret_cast<void *>(&tree_kernel<DH>);
    static std::mutex mu;
    static bool ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (dev >= 64 || !ready[dev]) {
            int most = 0;
            e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
            if (e != cudaSuccess) return e;
            if (dev < 64) ready[dev] = true;
        }
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(p.l.num_ctas);
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = p.l.smem_bytes;
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;
    void *args[] = {const_cast<TreeParams *>(&p)};
    (void)cudaGetLastError();
    e = cudaLaunchKernelExC(&lc, fn, args);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)p.rows.batch * p.rows.heads * p.n_tree * p.G;
    const int64_t blocks = (rows + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    lc.gridDim = dim3((unsigned)blocks);
    lc.blockDim = dim3(256);
    lc.dynamicSmemBytes = 0;
    return cudaLaunchKernelExC(&lc, reinterpret_cast<void *>(&tree_merge_kernel<DH>), args);
}

}  // namespace

bool plan_tree(const TreeParams &p, int max_smem, TreeLaunch *l)
{
    const int dh = p.dh;
    l->k_grouped = p.k.bits != 16 && p.k.group != dh;
    l->v_grouped = p.v.bits != 16 && p.v.group != dh;
    l->lo = (uint32_t)TT * dh * 2;
    l->k_bytes = l->lo * (l->k_grouped ? 2 : 1);
    l->v_bytes = l->lo * (l->v_grouped ? 2 : 1);
    const uint32_t kr = (uint32_t)TT * dh * p.k.bits / 8, vr = (uint32_t)TT * dh * p.v.bits / 8;
    const uint32_t pair = p.fmt == KVQ_FMT_ASYM ? 4 : 2;
    l->off_scales = std::max(kr, vr);
    const uint32_t ks = p.k.bits == 16 ? 0 : TT * (dh / p.k.group) * pair, vs = p.v.bits == 16 ? 0 : TT * (dh / p.v.group) * pair;
    l->entry_bytes = align_up(l->off_scales + std::max(ks, vs), 128);
    const uint32_t fixed = 1024 + TT * STAGE_LD * 4 + (uint32_t)sizeof(Par) + (uint32_t)sizeof(Ctl) + 512;
    // two converted tiles of K and of V where that leaves room for four raw ones
    for (int bufs = 2; bufs >= 1; bufs--) {
        l->k_bufs = bufs;
        l->v_bufs = bufs;
        const uint32_t conv = bufs * (l->k_bytes + l->v_bytes);
        if (fixed + conv + 2 * l->entry_bytes > (uint32_t)max_smem) continue;
        const uint32_t room = (uint32_t)max_smem - fixed - conv;
        l->entries = std::min<int>(kMaxEntries, room / l->entry_bytes);
        if (l->entries < 4 && bufs > 1) continue;
        if (l->entries < 2) continue;
        l->off_k = align_up((uint32_t)l->entries * l->entry_bytes, 1024);
        l->off_v = l->off_k + bufs * l->k_bytes;
        l->off_stage = l->off_v + bufs * l->v_bytes;
        l->off_par = align_up(l->off_stage + TT * STAGE_LD * 4, 16);
        l->off_ctl = align_up(l->off_par + (uint32_t)sizeof(Par), 16);
        l->smem_bytes = l->off_ctl + sizeof(Ctl) + 1024;
        return l->smem_bytes <= (size_t)max_smem;
    }
    return false;
}

cudaError_t launch_tree(const TreeParams &p, cudaStream_t stream)
{
    return p.dh == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace kvq
