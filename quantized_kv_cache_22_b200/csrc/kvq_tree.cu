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
// Roles of a CTA's 20 warps; nothing but barriers passes between them, each walks the segments
// by itself.
//   * A producer thread copies raw codes and scales (contiguous in either layout: one bulk
//     copy each) into a ring whose entries hold one tile of K or of V.
//   * Four warps turn K's codes, four V's, into f16 operands in 128-byte-swizzled shared
//     memory: every code (INT8, INT4, e4m3, code minus zero-point) is exact in f16.  One scale
//     per row stays outside the product.  Scales per group go in as x = code * (scale / 2^e) in
//     two f16 parts, hi = rn(x) and lo = x - hi (at most 8 + 11 significant bits), 2^e being a power
//     of two that brings the row's largest scale near f16's upper end; the product then takes both
//     parts.  Both are exact while a group's scale is within 2^21 of the row's largest (INT8 2^22,
//     INT4 2^26); below that its values are off by 2^-31 of the row's largest value at most.  e4m3's
//     small codes, whose last bit lies at 2^-9, are off by 2^-31 of the row's largest scale.
//   * One warp issues the products.  S = Q K^T: M = 128 rows, N = 128 tokens, A = Q in TMEM
//     (rows scaled by a power of two, fp32 rows in two parts), B = K, fp32 accumulators in TMEM,
//     S of even and of odd tiles apart.  O += P V: A = P in TMEM, B = V, MN-major.  (A from TMEM
//     takes 74 clocks a K step of 16 at N = 128, A from shared memory 107.)  The order is
//     S(i + 2), P V(i), so that the scores are two tiles ahead.
//   * Two softmax groups of four warps take the tiles in turns: a thread owns a TMEM lane.
//     z = s * scale_k + log2(scale_v) in log2 units, so that P = 2^(z - m) is the probability
//     times the value scale, rounded to f16 (the only rounding below fp32 in the path: the
//     product's other operand is f16 too; m keeps P between the subnormals and 2^14), and
//     l += P / scale_v in fp32.  O and m are common to both groups.  m moves only when a P would
//     pass 2^14; then O in TMEM is rescaled between two tiles' products, and a P that was made
//     with the older m is scaled by the power of two before it goes out.
//   * Few rows: with at most 64 (32) rows Q is laid into TMEM two (four) times, and each copy's
//     warps take one half (quarter) of the tile's tokens with zeros in the rest of their P, so
//     that all four warps share the exponentials; the copies' sums are joined at the end.
//     (64 rows: 119 us against 145 without copies; 32 rows: 160 against 266.)
//
// What bounds it.  16 x 8192 tokens of 8 KV heads, INT8, 4 heads a group: 114 to 121 us with 16
// drafted tokens (64 rows a KV head; its bytes alone would take 42), 276 to 292 with 64 (two row
// tiles, every tile converted for both; the products alone 84).  With 16, a tile of 128 tokens takes 3400
// cycles, of which the tensor cores work 1000 and the issue slots 1500 (conversion of 32
// thousand codes, 8 thousand exponentials); the rest is the chain scores - softmax - product of
// a tile, through three barriers of 100 cycles and more each.  Steps that measured well: K and V
// converted by warps of their own, 199 -> 144 us; two softmax groups, 144 -> 137; P in columns of
// its own and whole query rows in one load, 130 -> 125; a tile's scores in one product instead of
// two, 125 -> 113.  Groups that take tiles in turns instead of halves of each made short segments
// 5% faster.  A segment pays the opening of its row tile and its output, 8 to 12 thousand cycles
// with code and constants fetched cold, as much as three tiles, which the split over the CTAs does
// not count: of 64 sequences of up to 4000 tokens, INT4 in pages, 8 drafted, a CTA has 4.4 segments
// on average and 12 at most, 162 us; of 8 ragged ones of up to 2011, K INT8 and V INT4 in groups of
// 32, 24 drafted, 1.3 and 4, 49 us.  ptxas spills 716 bytes (880 with Dh 64) at the 96 registers that
// 640 threads leave.  Code of the same work moves the 64 sequences' time by 1 to 3%.
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
constexpr int kSoftWarps = 4, kConvWarps = 8;   // a softmax group's warps (two groups); converter warps
constexpr int kProducerWarp = 8, kMmaWarp = 9, kConvWarp0 = 12;   // (10 and 11 fill up their warpgroup)
constexpr int kThreads = 32 * (kConvWarp0 + kConvWarps);
constexpr int kConvThreads = 16 * kConvWarps;   // of K, and of V
constexpr int kMaxEntries = 12;
constexpr unsigned FULL = 0xffffffffu;

// Registers a thread: the block starts with 96 x 640 threads and shares them out anew by
// warpgroup (2 x softmax, producer and issuer, 2 x converters: 480 in all, as launched).
constexpr int kSoftRegs = 144, kIssueRegs = 64, kConvRegs = 64;
static_assert(2 * kSoftRegs + kIssueRegs + 2 * kConvRegs == 5 * 96, "the shares add up to the launch");
template <int N>
__device__ __forceinline__ void more_regs() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void fewer_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// TMEM columns: S of even and of odd tiles, O, Q (and the second part of fp32 queries), P
constexpr uint32_t COL_S = 0, COL_O = 256, COL_Q = 384, COL_QLO = 448, COL_P = 448;
constexpr uint32_t PANEL = TT * 128;    // 64 f16 of every token

// P in [0, 2^14]: m starts 6 to 7 below the first tile's maximum and follows when 14 is passed
constexpr float kHead = 6.f, kMoveAt = 14.f;

struct Work {
    long long n, u0;                    // all units, first unit of this CTA
    long long pre;                      // units before sequence b
    int p, n_units, b;                  // CTAs with work, units of this CTA, sequence of u0
};
struct Ctl {
    uint64_t full[kMaxEntries], empty[kMaxEntries];
    // by tile parity: a tile may have its scores (K converted, the S of two tiles before read,
    // queries in place); S done; V converted and P written; P V done
    uint64_t sready[2], sfull[2], pready[2], pvdone[2];
    uint64_t par[4], drain;             // V's per-token numbers of a tile are there (four deep)
    Work w;
    uint32_t tmem;
    int abort;
    float m[TT];                        // what O is scaled by, per TMEM lane
    alignas(16) float2 ml[TT][2];       // (m, l) of the groups
};
// Per-token numbers of a tile, four tiles deep: the converters run at most two tiles ahead of
// the softmax.
struct Par {
    float sk[4][TT], lv[4][TT], iv[4][TT];
};
template <int N>
struct Int {
    static constexpr int value = N;
};
constexpr int STAGE_BYTES = 2 * TT * 64;    // the epilogue's staging: 16 columns of a row by each group

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
// A launch parameter that a role uses in every tile, held in a register: left alone, the
// compiler reads it from the constant bank at each use, and a warp that runs alone waits there.
template <class X>
__device__ __forceinline__ X keep(X x)
{
    static_assert(sizeof(X) == 4, "one register");
    asm volatile("" : "+r"(x));
    return x;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Wait for the phase of the given parity, giving up after limit ns or when the abort flag is
// up.  A try returns at once when barriers change, which they do all the time in this kernel,
// and a waiting warp's tries take issue slots from the others: so it sleeps a little between
// them (NAP nanoseconds), longer where the role runs ahead of need anyway.
constexpr int kShortNap = 20, kLongNap = 100;
template <int NAP>
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, int parity, int *abort_flag, uint64_t limit)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (;;) {
#pragma unroll 1
        for (int n = 0; n < 64; n++) {
            if (mbar_try_wait(bar, parity & 1)) return true;
            __nanosleep(NAP);
        }
        const uint64_t t = globaltimer_ns();
        if (t0 == 0) t0 = t;
        if (*static_cast<volatile int *>(abort_flag) || t - t0 > limit) return false;
    }
}
// a wait of a whole warp: its lanes go on, or give up, together
template <int NAP>
__device__ __forceinline__ bool wait_warp(uint64_t *bar, int parity, int *abort_flag, uint64_t limit)
{
    return __all_sync(FULL, wait_bounded<NAP>(bar, parity, abort_flag, limit)) != 0;
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
#pragma unroll 1
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
#pragma unroll 1
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

// Walks the segments of the CTA: the tiles of one (sequence, KV head, row tile) that are its
// own.  Every role keeps its own walk, so that nothing but tiles passes between them.
struct Walk {
    int b, head, rt;                    // sequence, KV head, row tile
    int tile, count, left;              // first token tile, tiles of the segment, units left with it
    Seq s;
    __device__ __forceinline__ void start(const TreeParams &p, const Work &w)
    {
        left = w.n_units;
        count = 0;
        if (left == 0) return;
        b = w.b;
        s = sequence(p, b);
        const int off = (int)(w.u0 - w.pre), inner = off / s.tiles;
        tile = off - inner * s.tiles;
        head = inner / s.rtn;
        rt = inner - head * s.rtn;
        count = min(s.tiles - tile, left);
    }
    // the next segment; count 0: none is left
    __device__ __forceinline__ void next(const TreeParams &p)
    {
        left -= count;
        count = 0;
        if (left == 0) return;
        tile = 0;
        if (++rt == s.rtn) {
            rt = 0;
            if (++head == p.rows.heads) {
                head = 0;
#pragma unroll 1
                do s = sequence(p, ++b);
                while (s.tiles == 0);
            }
        }
        count = min(s.tiles, left);
    }
};

// ------------------------------------------------------------------ codes to f16
// log2 of what a value row whose scales are all zero gets for a scale: the token counts in the sum
// of the probabilities, but its P, which brings nothing, must not set m, or the others' P would fall
// among f16's subnormals.  Its codes are zeros too, as every append writes them; others would count
// 2^-64 each.  (Zeros in the operand instead took 2 to 10 % longer; and with a lower number ex2
// would flush a P to zero that l still needs.)
constexpr int kZeroRow = -64;

// Scales of one token as the converters see them.
struct RowScale {
    int e;        // exponent of the largest group scale (grouped)
    bool bad;     // a scale or zero-point that is not a finite number
    bool zero;    // every scale is zero
};
// Groups' factors scale / 2^e are raised by 2^kRaise, the most that keeps code * factor within f16
// (8 * 2^13, 127 * 2^9, 255 * 2^8, 448 * 2^7): a group whose scale is up to 2^(14 + kRaise) below its
// row's largest still has a normal f16 number for its factor.
template <int KIND>
constexpr int kRaise = KIND == K_INT4 ? 12 : KIND == K_INT8 ? 8 : KIND == K_ASYM ? 7 : 6;

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
    r.zero = m == 0;
    return r;
}

// A token's numbers: of K the factor of a score, of V log2 of the value scale (NaN where the
// row's values are not all numbers) and its inverse.
template <int KIND, bool GRP, bool ISV>
__device__ __forceinline__ void token_numbers(const uint16_t *sc, int t, bool bad, int nvalid, int ng, float tensor,
                                              bool is_tensor, float *p0, float *p1)
{
    constexpr int PAIR = KIND == K_ASYM ? 2 : 1;
    if constexpr (GRP) {
        const RowScale r = row_scale<KIND>(sc, t, ng);
        if constexpr (ISV) {
            const int e = r.zero ? kZeroRow : r.e - kRaise<KIND>;
            p0[t] = bad || r.bad ? __int_as_float(0x7fc00000) : (float)e;
            p1[t] = pow2i(-e);
        } else {
            p0[t] = pow2i(r.e - kRaise<KIND>);
        }
    } else {
        float s = 1.f;
        if (KIND != K_F16) s = is_tensor ? tensor : __half2float(__ushort_as_half(sc[t * PAIR]));
        if (KIND == K_ASYM) bad = bad || (sc[t * PAIR + 1] & 0x7fff) > 0x5bf8;
        if constexpr (ISV) {
            s = fabsf(s);
            if (!(s < INFINITY)) bad = true;
            // nothing may come of the token (the inverse meets P = 0 where it is masked, so it has
            // to be a number)
            if (bad || t >= nvalid) s = 1.f;
            if (s == 0.f) s = pow2i(kZeroRow);
            p0[t] = bad ? __int_as_float(0x7fc00000) : lg2(s);
            p1[t] = __fdividef(1.f, s);
        } else {
            p0[t] = s;
        }
    }
}

// One tile of K (ISV false) or V: raw codes and scales -> f16 operand rows.
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

    const uint8_t *src = raw + tr * ROW + c * Raw<KIND>::BYTES;
    uint8_t *out = dst + tr * 128 + ((c ^ tr) & 7) * 16;      // (t ^ tr) & 7 = 0: RPP is a multiple of 8
    uint32_t bad_rows = 0;                                     // CHECK: bit u for pass u
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
                float s = __half2float(__ushort_as_half(sc[(t * ng + g) * PAIR])) * pow2i(kRaise<KIND> - rs.e);
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
        for (int u = 0; u < PASSES; u++)
            token_numbers<KIND, GRP, ISV>(sc, u * RPP + tr, (bad_rows >> u) & 1u, nvalid, ng, tensor, is_tensor, p0, p1);
    if (__builtin_expect(ISV && nvalid < TT, 0)) {
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

// The converter role: every tile of K (ISV false) or V that is the CTA's, one kind of code per
// instance of the loop (a branch to the kind's code inside it would cost an instruction-cache
// miss on every tile: 2.1 against 1.5 thousand cycles a tile, INT8).
template <int DH, int KIND, bool GRP, bool ISV>
__device__ __forceinline__ bool convert_tiles(const TreeParams &p, const Work &w, uint8_t *smem, Ctl *ctl, Par *par,
                                              int ct, int *abort_flag, uint64_t limit)
{
    const CacheTensor &ten = ISV ? p.v : p.k;
    const int ng = keep(DH / ten.group), gshift = ten.group == 32 ? 5 : ten.group == 64 ? 6 : 7;
    const bool is_tensor = keep(p.fmt) == KVQ_FMT_TENSOR;
    const float tensor = is_tensor ? __half2float(ten.scales[0]) : 1.f;
    const int bufs = keep(ISV ? p.l.v_bufs : p.l.k_bufs), E = keep(p.l.entries);
    uint8_t *tiles = smem + keep(ISV ? p.l.off_v : p.l.off_k);
    const uint32_t tile_bytes = keep(ISV ? p.l.v_bytes : p.l.k_bytes), entry_bytes = keep(p.l.entry_bytes);
    const uint32_t off_scales = keep(p.l.off_scales), lo = keep(p.l.lo);
    uint64_t *ready = ISV ? ctl->pready : ctl->sready, *used = ISV ? ctl->pvdone : ctl->sfull;
    constexpr bool CHECK = ISV && (KIND == K_E4M3 || KIND == K_F16);   // numbers after the conversion
    int s = ISV, use = 0, i = 0;
    Walk it;
#pragma unroll 1
    for (it.start(p, w); it.count; it.next(p)) {
        int left = it.s.total - it.tile * TT;
#pragma unroll 1
        for (int k = it.count; k > 0; k--, i++, left -= TT) {
            if (!wait_warp<kLongNap>(&ctl->full[s], use, abort_flag, limit)) return false;
            const uint8_t *entry = smem + (uint32_t)s * entry_bytes;
            const uint16_t *sc = reinterpret_cast<const uint16_t *>(entry + off_scales);
            float *p0 = ISV ? par->lv[i & 3] : par->sk[i & 3], *p1 = par->iv[i & 3];
            if (ISV && !CHECK) {
                // V's numbers before its buffer is free: the softmax wants them that much earlier
                // (slot i & 3 was last read for tile i - 4, whose P V is done)
                token_numbers<KIND, GRP, ISV>(sc, ct, false, min(TT, left), ng, tensor, is_tensor, p0, p1);
                __syncwarp();
                mbar_arrive_if(&ctl->par[i & 3], (ct & 31) == 0);
            }
            // the operand's last use: S, or P V, of tile i - bufs
            if (i >= bufs && !wait_warp<kLongNap>(&used[(i - bufs) & 1], (i - bufs) >> 1, abort_flag, limit)) return false;
            // (S of tile i - 2 is done, so that its group has read the numbers of tile i - 4)
            if (!ISV) token_numbers<KIND, GRP, ISV>(sc, ct, false, min(TT, left), ng, tensor, is_tensor, p0, p1);
            convert<DH, KIND, GRP, ISV>(entry, sc, tiles + (uint32_t)(i & (bufs - 1)) * tile_bytes, lo, min(TT, left), ct, ng,
                                        gshift, tensor, is_tensor, p0, p1);
            fence_proxy_async_shared();
            __syncwarp();
            if (CHECK) mbar_arrive_if(&ctl->par[i & 3], (ct & 31) == 0);
            mbar_arrive_if(&ready[i & 1], (ct & 31) == 0);
            mbar_arrive_if(&ctl->empty[s], (ct & 31) == 0);
            s += 2;
            if (s >= E) {
                s -= E;
                ++use;
            }
        }
    }
    return true;
}

template <int DH, bool ISV>
__device__ __forceinline__ bool convert_role(const TreeParams &p, const Work &w, uint8_t *smem, Ctl *ctl, Par *par,
                                             int ct, int *abort_flag, uint64_t limit)
{
    const bool grp = ISV ? p.l.v_grouped : p.l.k_grouped;
    switch (kind_of(ISV ? p.v.bits : p.k.bits, p.fmt) * 2 + grp) {
    case 2 * K_INT8: return convert_tiles<DH, K_INT8, false, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_INT8 + 1: return convert_tiles<DH, K_INT8, true, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_INT4: return convert_tiles<DH, K_INT4, false, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_INT4 + 1: return convert_tiles<DH, K_INT4, true, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_E4M3: return convert_tiles<DH, K_E4M3, false, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_E4M3 + 1: return convert_tiles<DH, K_E4M3, true, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_ASYM: return convert_tiles<DH, K_ASYM, false, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    case 2 * K_ASYM + 1: return convert_tiles<DH, K_ASYM, true, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    default: return convert_tiles<DH, K_F16, false, ISV>(p, w, smem, ctl, par, ct, abort_flag, limit);
    }
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

// z of N tokens (scores, fp32 accumulators in a, times the row's and the tokens' factors,
// plus log2 of the value scales; -inf where the row does not look), and their maximum
template <int N>
__device__ __forceinline__ float scores(const uint32_t (&a)[N], const float *sk, const float *lv, float rf,
                                        uint32_t vis, uint64_t (&z)[N / 2])
{
    const uint64_t rf2 = pair(rf, rf);
#pragma unroll
    for (int t = 0; t < N / 2; t += 2) {
        const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(sk + 2 * t);
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(lv + 2 * t);
        z[t] = fma2(mul2(pair(a[2 * t], a[2 * t + 1]), k.x), rf2, v.x);
        z[t + 1] = fma2(mul2(pair(a[2 * t + 2], a[2 * t + 3]), k.y), rf2, v.y);
    }
    if (__builtin_expect(vis != FULL, 0)) {
#pragma unroll
        for (int t = 0; t < N / 2; t++)
            z[t] = pair((vis >> (2 * t)) & 1u ? first(z[t]) : -INFINITY,
                        (vis >> (2 * t + 1)) & 1u ? second(z[t]) : -INFINITY);
    }
    float m0 = fmaxf(first(z[0]), second(z[0])), m1 = fmaxf(first(z[1]), second(z[1]));
#pragma unroll
    for (int t = 2; t < N / 2; t += 2) {
        m0 = fmaxf(m0, fmaxf(first(z[t]), second(z[t])));
        m1 = fmaxf(m1, fmaxf(first(z[t + 1]), second(z[t + 1])));
    }
    return fmaxf(m0, m1);
}

// P = 2^(z - m) of N tokens, rounded to f16, into N / 2 packed columns; returns their share of l
template <int N>
__device__ __forceinline__ float probs(const uint64_t (&z)[N / 2], const float *iv, float m, uint32_t (&w)[N / 2])
{
    const uint64_t nm = pair(-m, -m);
    uint64_t l0 = 0, l1 = 0;
#pragma unroll
    for (int t = 0; t < N / 2; t += 2) {
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
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + keep(p.l.off_ctl));
    Par *par = reinterpret_cast<Par *>(smem + keep(p.l.off_par));
    int *abort_flag = &ctl->abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = keep(p.l.entries), KB = keep(p.l.k_bufs), VB = keep(p.l.v_bufs);
    const uint64_t limit = p.timeout_ns;
    auto give_up = [&]() {
        *static_cast<volatile int *>(abort_flag) = 1;
        atomicExch(p.status, KVQ_ERR_TIMEOUT);
    };
    auto wait1 = [&](uint64_t *bar, int parity) { return wait_bounded<kShortNap>(bar, parity, abort_flag, limit); };
    auto wait = [&](uint64_t *bar, int parity) { return wait_warp<kShortNap>(bar, parity, abort_flag, limit); };

    if (threadIdx.x == 0) {
        for (int s = 0; s < E; s++) {
            mbar_init(&ctl->full[s], 1);
            mbar_init(&ctl->empty[s], kConvWarps / 2);
        }
        for (int j = 0; j < 2; j++) {
            mbar_init(&ctl->sready[j], kConvWarps / 2 + kSoftWarps);
            mbar_init(&ctl->sfull[j], 1);
            mbar_init(&ctl->pready[j], kConvWarps / 2 + kSoftWarps);
            mbar_init(&ctl->pvdone[j], 1);
        }
        for (int j = 0; j < 4; j++) mbar_init(&ctl->par[j], kConvWarps / 2);
        mbar_init(&ctl->drain, 1);
        ctl->abort = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < TT) ctl->m[threadIdx.x] = -INFINITY;
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
    // P has columns of its own, unless the second part of fp32 queries takes them: then it lies
    // over its scores, which then wait for it
    const bool over = keep(p.q_dtype) == KVQ_F32;

    if (warp < 2 * kSoftWarps) {
        more_regs<kSoftRegs>();
        // ====================== softmax ======================
        // two groups of four warps take the tiles in turns (a tile's scores are in the S of its
        // parity); O, and the m that it is scaled by, are common to both
        const int grp = warp / kSoftWarps;
        const int place = threadIdx.x & (TT - 1);    // TMEM lane
        const uint32_t lane_off = (uint32_t)(place & ~31) << 16;
        const uint32_t s_row = tmem + COL_S + 128u * grp + lane_off, o_row = tmem + COL_O + lane_off;
        const uint32_t p_row = over ? s_row : tmem + COL_P + lane_off;
        float4 *stage = reinterpret_cast<float4 *>(smem + keep(p.l.off_stage));
        float osign = 1.f;
        if (p.fmt == KVQ_FMT_TENSOR) {
            const float s = __half2float(p.v.scales[0]);
            osign = s < 0.f ? -1.f : s == 0.f ? 0.f : 1.f;
        }
        // A wait that gave up does not end the role: the eight warps meet at a hardware barrier
        // at every segment's end, so all of them walk on to the end (with the abort flag up no
        // further wait takes time) and write nothing more.
        bool ok = true;
        auto hold = [&](uint64_t *bar, int parity) {
            if (__builtin_expect(!mbar_try_wait(bar, parity & 1), 0))
                if (!wait1(bar, parity) && ok) {
                    ok = false;
                    give_up();
                }
            __syncwarp();
        };
        auto soft_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(64 * kSoftWarps) : "memory"); };
        // What a thread keeps of its row; the next segment's is made while the last tile of the
        // current one is with the tensor cores.
        struct Row {
            int rows, copies, tb;                    // rows of the tile, their copies; first token of a tile
                                                     // that this copy takes
            float rf;                                // factor of a score: tau log2(e), the query's power of two
            uint64_t mask;                           // drafted tokens that the row attends
        };
        // this thread's row of the walk's segment; store: its query into TMEM
        // (once free_q() says that the scores of the segment before are done)
        auto open = [&](const Walk &o, bool store, auto &&free_q) {
            Row x;
            x.rows = min(kTreeRows, o.s.n * p.G - o.rt * kTreeRows);
            x.copies = x.rows <= 32 ? 4 : x.rows <= 64 ? 2 : 1;
            const int r = place & (TT / x.copies - 1);
            x.tb = place - r;
            const int rr = o.rt * kTreeRows + r, qi = rr / p.G;
            const bool live = r < x.rows;
            const int64_t at = (((int64_t)o.b * p.n_tree + qi) * p.n_q_heads + (int64_t)o.head * p.G + rr - qi * p.G) * DH;
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
            if (p.q_dtype == KVQ_F16 && !store) return x;
            // (loops kept rolled: this runs once a segment, and code that is not in the
            // instruction cache takes longer to fetch than to run)
            if (p.q_dtype != KVQ_F32) {
                const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at);
                const uint4 none = make_uint4(0u, 0u, 0u, 0u);
                float pre = 1.f;
                if (p.q_dtype == KVQ_BF16) {
                    uint32_t top = 0u;                              // (bf16 magnitudes compare as integers)
#pragma unroll 1
                    for (int c = 0; c < DH / 8; c += 8) {
                        uint4 u[8];
#pragma unroll
                        for (int k = 0; k < 8; k++) u[k] = live ? src[c + k] : none;
#pragma unroll
                        for (int k = 0; k < 8; k++) {
                            top = __vmaxu2(top, __vmaxu2(u[k].x & 0x7fff7fffu, u[k].y & 0x7fff7fffu));
                            top = __vmaxu2(top, __vmaxu2(u[k].z & 0x7fff7fffu, u[k].w & 0x7fff7fffu));
                        }
                    }
                    pre = level(__uint_as_float(max(top & 0xffff0000u, top << 16)));
                    if (!store) return x;
                }
                free_q();
#pragma unroll 1
                for (int c = 0; c < DH / 32; c++) {
                    uint4 u[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) u[k] = live ? src[4 * c + k] : none;
                    uint32_t *h = reinterpret_cast<uint32_t *>(u);
                    if (p.q_dtype == KVQ_BF16)
#pragma unroll
                        for (int k = 0; k < 16; k++)
                            h[k] = pack_half2(__uint_as_float(h[k] << 16) * pre, __uint_as_float(h[k] & 0xffff0000u) * pre);
                    tmem_st16(tmem + COL_Q + lane_off + 16u * c, *reinterpret_cast<uint32_t(*)[16]>(h));
                }
            } else {
                const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at);
                const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
                float a = 0.f;
#pragma unroll 8
                for (int k = 0; k < DH / 4; k++) {
                    const float4 f = live ? src[k] : none;
                    a = fmaxf(fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
                }
                const float pre = level(a);
                if (!store) return x;
                free_q();
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
            return x;
        };
        Walk it;
        Row row{};
        float m = -INFINITY, l = 0.f;                // the group's: l in units of 2^m
        int i = 0;                                   // units done
        // P of tile i, CH times 32 tokens a thread.
        // The probabilities are made in registers, with the m that the group's tile before ended with
        // (the other group may have raised it already or not: bits must not depend on that).
        // P's columns are free, and m is final up to this tile, once P V of the tile before is
        // done: then P goes out, scaled again if the other group has raised m meanwhile.
        // m is raised in a second pass over the tile, when some token would not fit; O is then
        // rescaled between the two tiles' P V, with no other P in flight.
        auto tiles = [&](auto ch, int i0, int count) {
            constexpr int CH = decltype(ch)::value, N = 32;
#pragma unroll 1
            for (int k = (i0 ^ grp) & 1; k < count; k += 2) {
                i = i0 + k;
                const int j = i & 1;                     // == grp
                const float *sk = par->sk[i & 3] + row.tb, *lv = par->lv[i & 3] + row.tb, *iv = par->iv[i & 3] + row.tb;
                const int t0 = (it.tile + k) * TT + row.tb;
                const bool whole = t0 + 32 * CH <= it.s.len;
                const uint32_t s_at = s_row + (uint32_t)row.tb, p_at = p_row + (uint32_t)row.tb / 2;
                uint32_t pw[CH][16];
                float sum;
                hold(&ctl->sfull[j], i >> 1);
                hold(&ctl->par[i & 3], i >> 2);
                tc_fence_after();
#pragma unroll 1
                for (bool second = false;; second = true) {
                    bool fits = true;
                    sum = 0.f;
                    const float me = m == -INFINITY ? 0.f : m;
#pragma unroll
                    for (int c = 0; c < 32 * CH; c += N) {
                        uint32_t a[N];
                        uint64_t z[N / 2];
                        tmem_ld_async(s_at + c, a);
                        tmem_ld_wait(a);
                        const uint32_t vis = whole ? FULL : visible(t0 + c, it.s.len, row.mask);
                        const float mx = scores<N>(a, sk + c, lv + c, row.rf, vis, z);
                        fits = fits && (!(mx > m + kMoveAt) || mx == -INFINITY);
                        sum += probs<N>(z, iv + c, me, pw[c / N]);
                    }
                    if (second || __builtin_expect(__all_sync(FULL, fits), 1)) break;
                    // ---- the tile's maximum, then m, O and l after it
                    float top = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 32 * CH; c += 16) {
                        uint32_t a[16];
                        uint64_t z[8];
                        tmem_ld_async(s_at + c, a);
                        tmem_ld_wait(a);
                        const uint32_t vis = whole ? FULL : visible(t0 + c, it.s.len, row.mask) | 0xffff0000u;
                        top = fmaxf(top, scores<16>(a, sk + c, lv + c, row.rf, vis, z));
                    }
                    if (k > 0) hold(&ctl->pvdone[j ^ 1], (i - 1) >> 1);
                    tc_fence_after();
                    const float was = ctl->m[place];
                    const bool set = was == -INFINITY && top > -INFINITY, up = !set && top > was + kMoveAt;
                    const float to = set || up ? floorf(top) - kHead : was;
                    const float alpha = up ? ex2(was - to) : 1.f;     // both whole: a power of two
                    if (__any_sync(FULL, up)) {
#pragma unroll 1
                        for (int q = 0; q < DH; q += 16) {
                            uint32_t x[16];
                            tmem_ld16(o_row + q, x);
#pragma unroll
                            for (int y = 0; y < 16; y++) x[y] = __float_as_uint(__uint_as_float(x[y]) * alpha);
                            tmem_st16(o_row + q, x);
                        }
                    }
                    ctl->m[place] = to;
                    if (to != m) {
                        l *= ex2(m - to);
                        m = to;
                    }
                }
                l += sum;
                // the scores are read: those of two tiles on may come
                if (!over && k + 2 < count) {
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_if(&ctl->sready[j], lane == 0);
                }
                if (k > 0) hold(&ctl->pvdone[j ^ 1], (i - 1) >> 1);
                tc_fence_after();
                const float then = ctl->m[place];
                if (__builtin_expect(__any_sync(FULL, then != m), 0)) {
                    // a power of two, in two factors: f16 holds them down to 2^-24 (of a P below 2^14
                    // nothing is left beyond 2^-48, and an m of -inf has left zeros)
                    float d = m == then ? 0.f : m - then;
                    l *= ex2(d);
                    m = then;
                    d = fmaxf(d, -48.f);
#pragma unroll 1
                    for (int k2 = 0; k2 < 2; k2++) {
                        const float alpha = ex2(fmaxf(d, -24.f));
                        const uint32_t alpha2 = pack_half2(alpha, alpha);
                        d -= fmaxf(d, -24.f);
#pragma unroll
                        for (int c = 0; c < CH; c++)
#pragma unroll
                            for (int q = 0; q < 16; q++) pw[c][q] = hmul2_u32(pw[c][q], alpha2);
                    }
                }
#pragma unroll
                for (int c = 0; c < CH; c++) tmem_st16(p_at + 16u * c, pw[c]);
                if (CH < 4 && (over || k == 0)) {
                    // zeros for the other copies' tokens: scores left theirs, or the tile is the first
                    uint32_t none[16];
#pragma unroll
                    for (int x = 0; x < 16; x++) none[x] = 0u;
#pragma unroll 1
                    for (int c = CH; c < 4; c++) tmem_st16(p_row + (((uint32_t)row.tb / 2 + 16u * c) & 63u), none);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                mbar_arrive_if(&ctl->pready[j], lane == 0);
                if (over && k + 2 < count) mbar_arrive_if(&ctl->sready[j], lane == 0);
            }
        };
        // segment by segment; a first pass without tiles only opens the first one
        it.start(p, w);
        bool opened = false;
#pragma unroll 1
        while (it.count) {
            const int i0 = i, copies = row.copies, count = opened ? it.count : 0;
            if (copies == 1)
                tiles(Int<4>(), i0, count);
            else if (copies == 2)
                tiles(Int<2>(), i0, count);
            else
                tiles(Int<1>(), i0, count);
            i = i0 + count;
            // ---- the next segment's queries come in, by the group of its first tile, once this
            // one's scores are all done; the other group has read its S
            const int last = i - 1;
            Walk ahead = it;
            if (opened) ahead.next(p);
            Row next{};
            if (ahead.count) {
                const bool mine = (i & 1) == grp;
                next = open(ahead, mine, [&]() {
                    if (!opened) return;
                    hold(&ctl->sfull[last & 1], last >> 1);
                    tc_fence_after();
                });
                tc_fence_before();
                __syncwarp();
                if (mine || ahead.count > 1) mbar_arrive_if(&ctl->sready[grp], lane == 0);
            }
            if (!opened) {
                opened = true;
                row = next;
                continue;
            }
            // ---- join the groups' sums and the copies of every row; the output, or a partial
            const int nr = TT / copies, r = place & (nr - 1), rows = row.rows;
            const bool direct = it.tile == 0 && it.count == it.s.tiles;
            // a CTA leaves two partials at most: of its first segment, and of its last
            float *part = p.slots + (int64_t)(2 * (int)blockIdx.x + (i0 == 0 ? 0 : 1)) * tree_slot_floats(p.slot_rows, DH);
            float *part_ml = part + (int64_t)p.slot_rows * DH + 2 * place;
            int64_t out0 = ((int64_t)it.b * p.n_tree * p.n_q_heads + (int64_t)it.head * p.G) * DH;
            float per_g = 1.f / (float)p.G;
            int out_dtype = p.out_dtype, q_gap = p.n_q_heads - p.G;
            // (all of it before the wait)
            asm volatile("" : "+l"(part), "+l"(part_ml), "+l"(out0), "+f"(per_g), "+r"(out_dtype), "+r"(q_gap));
            // where row rr of the tile goes
            auto row_at = [&](int rr) {
                const int gr = it.rt * kTreeRows + rr;
                return out0 + ((int64_t)(int)(((float)gr + 0.5f) * per_g) * q_gap + gr) * DH;
            };
            ctl->ml[place][grp] = make_float2(m, l);
            hold(&ctl->pvdone[last & 1], last >> 1);
            tc_fence_after();
            soft_sync();
            float4 x[4];                                             // m, l of a copy from either group
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                x[c] = c < copies ? *reinterpret_cast<const float4 *>(ctl->ml[r + c * nr])
                                  : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
                M = fmaxf(M, fmaxf(x[c].x, x[c].z));
            }
#pragma unroll
            for (int c = 0; c < 4; c++) {
                L += x[c].x == -INFINITY ? 0.f : x[c].y * ex2(x[c].x - M);
                L += x[c].z == -INFINITY ? 0.f : x[c].w * ex2(x[c].z - M);
            }
            const float mine = fmaxf(ctl->ml[place][0].x, ctl->ml[place][1].x);     // what O is scaled by
            if (grp == 0) ctl->m[place] = -INFINITY;                 // for the next segment
            float f = mine == -INFINITY ? 0.f : ex2(mine - M) * osign;
            if (direct) f = L != 0.f ? f / L : 0.f;
            if (!direct && ok && threadIdx.x < rows) *reinterpret_cast<float2 *>(part_ml) = make_float2(M, L);
            if (copies == 1) {
                // every thread has a row's sums: half of its columns, 16 a time (through the
                // staging below 8 x 2011 tokens, 72 rows, took 52.4 us, so 50.8)
                const int64_t at = (direct ? row_at(place) : (int64_t)place * DH) + DH / 2 * grp;
#pragma unroll 1
                for (int c = 0; c < DH / 2; c += 16) {
                    uint32_t o[16];
                    tmem_ld16(o_row + c + DH / 2 * grp, o);
                    float y[16];
#pragma unroll
                    for (int k = 0; k < 16; k++) y[k] = f == 0.f ? 0.f : __uint_as_float(o[k]) * f;
                    if (place < rows && ok) {
                        if (direct) {
                            store8(p.out, at + c, out_dtype, *reinterpret_cast<float(*)[8]>(y));
                            store8(p.out, at + c + 8, out_dtype, *reinterpret_cast<float(*)[8]>(y + 8));
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; k++) reinterpret_cast<float4 *>(part + at + c)[k] = reinterpret_cast<float4 *>(y)[k];
                        }
                    }
                }
                soft_sync();
            } else {
                // 32 columns of O a round, 16 by each group; then eight lanes a row, four columns
                // each.  Staged rows are 64 bytes, their 16-byte pieces permuted so that neither
                // side meets bank conflicts.
                const int r0 = threadIdx.x >> 3, half = (threadIdx.x >> 2) & 1, piece = threadIdx.x & 3;
                float4 *put = stage + (grp * TT + (place ^ grp)) * 4;
                const int put_x = (place >> 1) & 3;
#pragma unroll 1
                for (int c = 0; c < DH; c += 32) {
                    uint32_t o[16];
                    tmem_ld16(o_row + c + 16u * grp, o);
#pragma unroll
                    for (int k = 0; k < 16; k++) o[k] = f == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * f);
                    if (c > 0) soft_sync();                          // the staging was read
#pragma unroll
                    for (int k = 0; k < 4; k++) put[k ^ put_x] = reinterpret_cast<float4 *>(o)[k];
                    soft_sync();
#pragma unroll 1
                    for (int rr = r0; rr < rows && ok; rr += 32) {
                        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            if (k >= copies) break;
                            const int q = rr + k * nr;
                            const float4 v = stage[(half * TT + (q ^ half)) * 4 + (piece ^ ((q >> 1) & 3))];
                            y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
                        }
                        const int at = c + 16 * half + 4 * piece;
                        if (direct)
                            store4(p.out, row_at(rr) + at, out_dtype, y);
                        else
                            *reinterpret_cast<float4 *>(part + rr * DH + at) = make_float4(y[0], y[1], y[2], y[3]);
                    }
                }
            }
            m = -INFINITY;
            l = 0.f;
            row = next;
            it = ahead;
        }
    } else if (warp >= kConvWarp0) {
        fewer_regs<kConvRegs>();
        // ====================== converters ======================
        // four warps turn K tiles, four V tiles
        const int ct = (threadIdx.x - 32 * kConvWarp0) & (kConvThreads - 1);
        const bool ok = warp < kConvWarp0 + kConvWarps / 2
                            ? convert_role<DH, false>(p, w, smem, ctl, par, ct, abort_flag, limit)
                            : convert_role<DH, true>(p, w, smem, ctl, par, ct, abort_flag, limit);
        if (!ok) give_up();
    } else {
        fewer_regs<kIssueRegs>();
        if (warp == kProducerWarp && lane == 0) {
            // ====================== producer ======================
            const uint64_t pol = l2_evict_first_policy();
            const int kr = DH * p.k.bits / 8, vr = DH * p.v.bits / 8;
            const bool sc = p.fmt != KVQ_FMT_TENSOR;
            const int ksb = sc && p.k.bits != 16 ? DH / p.k.group * scale_vals(p.fmt) * 2 : 0;   // 0: no scales
            const int vsb = sc && p.v.bits != 16 ? DH / p.v.group * scale_vals(p.fmt) * 2 : 0;
            int e = 0, s = 0, use = 0;          // entries filled; the next one's place and use
            bool ok = true;
            int serve = p.serve;                // segments to copy (self-test: the rest is withheld)
            Walk it;
#pragma unroll 1
            for (it.start(p, w); it.count && ok; it.next(p)) {
                if (serve-- <= 0) break;
#pragma unroll 1
                for (int t = it.tile; t < it.tile + it.count && ok; t++) {
                    const int nv = min(TT, it.s.total - t * TT);
                    int64_t row;
                    if (p.rows.block_table != nullptr) {
                        int page = p.rows.block_table[(int64_t)it.b * p.rows.max_pages + t];
                        page = min(max(page, 0), p.rows.n_pages - 1);   // stay inside the pool
                        row = ((int64_t)page * p.rows.heads + it.head) * kPageTokens;
                    } else {
                        row = ((int64_t)it.b * p.rows.heads + it.head) * p.rows.cap + t * TT;
                    }
                    const int nsc = (nv + 7) & ~7;      // rows whose scales are whole 16-byte pieces
#pragma unroll 1
                    for (int kv = 0; kv < 2; kv++, e++) {
                        if (use > 0 && !(ok = wait_bounded<kLongNap>(&ctl->empty[s], use - 1, abort_flag, limit))) break;
                        const CacheTensor &ten = kv ? p.v : p.k;
                        const int rb = kv ? vr : kr, sb = kv ? vsb : ksb;
                        uint8_t *dst = smem + (uint32_t)s * p.l.entry_bytes;
                        mbar_arrive_expect_tx(&ctl->full[s], (uint32_t)(nv * rb + nsc * sb));
                        bulk_load_hint(dst, ten.codes + row * rb, (uint32_t)(nv * rb), &ctl->full[s], pol);
                        if (sb)
                            bulk_load_hint(dst + p.l.off_scales, reinterpret_cast<const uint8_t *>(ten.scales) + row * sb,
                                           (uint32_t)(nsc * sb), &ctl->full[s], pol);
                        if (++s == E) {
                            s = 0;
                            ++use;
                        }
                    }
                }
            }
            if (!ok) give_up();
            // copies in flight land before the CTA ends, whatever the other roles did
#pragma unroll 1
            for (int k = e > E ? e - E : 0; k < e; k++) (void)mbar_wait_drain(&ctl->full[k % E], (k / E) & 1, limit);
        } else if (warp == kMmaWarp && n_units > 0) {
            // ====================== MMA issuer ======================
            // The whole warp walks, so that every operand is the same for all its lanes and stays
            // in uniform registers; one lane issues.
            const bool leader = elect_one();
            const uint32_t tm = __shfl_sync(FULL, tmem, 0);
            const uint32_t sbase = smem_u32(smem);
            const uint64_t k_desc = sw128_desc(sbase + keep(p.l.off_k)), v_desc = sw128_mn_desc(sbase + keep(p.l.off_v), PANEL, 1024u);
            // (descriptors count 16-byte units)
            const uint32_t lo = keep(p.l.lo) >> 4, k_step = keep(p.l.k_bytes) >> 4, v_step = keep(p.l.v_bytes) >> 4;
            const int q_parts = over ? 2 : 1, s_parts = (1 + keep(p.l.k_grouped)) * q_parts, v_parts = 1 + keep(p.l.v_grouped);
            // scores of tile i
            auto issue_s = [&](int i) {
                if (!wait(&ctl->sready[i & 1], i >> 1)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int part = 0; part < s_parts; part++) {
                    const int kp = q_parts == 2 ? part >> 1 : part, qp = q_parts == 2 ? part & 1 : 0;
                    const uint64_t d = k_desc + ((i & (KB - 1)) * k_step + kp * lo);
                    const uint32_t qa = tm + (qp ? COL_QLO : COL_Q), st = tm + COL_S + 128u * (i & 1);
                    if (leader)
#pragma unroll
                        for (int kk = 0; kk < DH / 16; kk++)
                            umma_f16_ts(st, qa + 8u * kk, d + ((kk >> 2) * (PANEL >> 4) + 2u * (kk & 3)), IDESC_S,
                                        kk > 0 ? 1u : (uint32_t)(part > 0));
                }
                if (leader) umma_commit(&ctl->sfull[i & 1]);
                __syncwarp();
                return true;
            };
            // O += P V of tile i
            auto issue_pv = [&](int i, bool first) {
                if (!wait(&ctl->pready[i & 1], i >> 1)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int part = 0; part < v_parts; part++) {
                    const uint64_t d = v_desc + ((i & (VB - 1)) * v_step + part * lo);
                    const uint32_t pa = tm + (over ? COL_S + 128u * (i & 1) : COL_P);
                    if (leader)
#pragma unroll
                        for (int kk = 0; kk < TT / 16; kk++)
                            umma_f16_ts(tm + COL_O, pa + 8u * kk, d + 128u * kk, IDESC_O,
                                        kk > 0 ? 1u : (uint32_t)(!first || part > 0));
                }
                if (leader) umma_commit(&ctl->pvdone[i & 1]);
                __syncwarp();
                return true;
            };
            int i = 0;
            bool ok = true;
            Walk it;
#pragma unroll 1
            for (it.start(p, w); it.count && ok; it.next(p)) {
                const int count = __shfl_sync(FULL, it.count, 0);
                ok = issue_s(i) && (count < 2 || issue_s(i + 1));
#pragma unroll 1
                for (int k = 0; k < count && ok; k++, i++) {
                    // scores two tiles ahead, over those that are read: before this tile's P V,
                    // unless its P lies there
                    const bool more = k + 2 < count;
                    if (more && !over) ok = issue_s(i + 2);
                    ok = ok && issue_pv(i, k == 0);
                    if (more && over) ok = ok && issue_s(i + 2);
                }
            }
            if (!ok) give_up();
            // every product issued completes before the CTA gives up its memory
            if (leader) {
                umma_commit(&ctl->drain);
                (void)mbar_wait_drain(&ctl->drain, 0, limit);
            }
            __syncwarp();
        } else if (warp == kMmaWarp + 1 && lane == 0) {
            // ====================== where the partials are ======================
            // of every row tile whose first tokens are this CTA's: the slot of its first partial,
            // the CTA, how many CTAs share it
            Walk it;
            int done = 0;
#pragma unroll 1
            for (it.start(p, w); it.count; it.next(p)) {
                if (it.tile == 0)
                    p.seg[((int64_t)it.b * p.rows.heads + it.head) * p.row_tiles + it.rt] =
                        make_int4(2 * (int)blockIdx.x + (done == 0 ? 0 : 1), blockIdx.x,
                                  it.count == it.s.tiles ? 1 : range_cta(w.u0 + done + it.s.tiles - 1, w.n, w.p) - (int)blockIdx.x + 1, 0);
                done += it.count;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

// One warp joins the partials of one row whose row tile several CTAs shared: bound by latency
// (the row tile's entry, the maxima, then the sums), 4 to 14 us apart from the kernel before,
// most of it launch and cold fetches.
template <int DH>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeParams p)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const unsigned blocks = (unsigned)(p.n_tree * p.G + 7) / 8, at_bh = blockIdx.x / blocks;
    const int rr = (int)(blockIdx.x - at_bh * blocks) * 8 + (int)(threadIdx.x >> 5);
    const int b = (int)(at_bh / (unsigned)p.rows.heads), head = (int)(at_bh - (unsigned)b * (unsigned)p.rows.heads);
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
#pragma unroll 2
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
    e = launch_dependent(tree_kernel<DH>, (unsigned)p.l.num_ctas, kThreads, p.l.smem_bytes, stream, p);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (int64_t)p.rows.batch * p.rows.heads * ((p.n_tree * p.G + 7) / 8);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(tree_merge_kernel<DH>, (unsigned)blocks, 256, 0, stream, p);
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
    const uint32_t fixed = 1024 + STAGE_BYTES + (uint32_t)sizeof(Par) + (uint32_t)sizeof(Ctl) + 512;
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
        l->off_par = align_up(l->off_stage + STAGE_BYTES, 16);
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
