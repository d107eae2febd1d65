// sparse_attn_fp4.cu -- sparse_attn over a paged cache of 4-bit rows, on 8-bit tensor-core operands.
//
// "Module attn", sparse_attn and the Precision paragraph: softmax over the index-listed rows of the shared
// latent tensor with a sink in the denominator, the rows reused as values, f32 arithmetic, bf16 output;
// "DeepSeek V4.1", attention/query-latent, Attention.forward (the output's inverse rotation).  Rows are
// e2m1 codes with a power-of-two scale per 32 values, reached through a table of pages.
//
// The mathematics.  A row is v_r = 2^(e_r - 12) c_r, e_r its largest block exponent, -96 at least, and c_r its codes
// times 2^(k - e_r + 12): e2m1 has one mantissa bit, so c_r is exact in e5m2 for blocks down to 26 octaves below
// e_r (lower ones count as zeros).  Exponents above 100 are read as 100 and flagged: with e_r in [-96, 100] the scores'
// products (2^32 2^(e_r - 12)) and the sums of P' 2^-e_r (of 2^20 rows) stay below f32's largest.
// One byte a value serves as key and as value, and the row's own power of two moves to where the row is a
// single number: to its scores, and to its probability.
//  * q = 2^g (hi + 2^-5 lo), hi and lo in e4m3: hi holds q's top four significant bits, lo the four below
//    them, so a bf16 q (eight) is exact down to 2^-9 of its head's largest value and off by 2^-22 of that
//    largest value below.  S^T = C [hi | lo]: M = 128 rows, N = 64 heads twice, and the score is
//    (S_hi + 2^-5 S_lo) 2^(g + e_r - 12) scale.
//  * P' = 2^(s + e_r - m + 4), m the head's running maximum of s + e_r (lazily raised, at most 4 octaves late),
//    at most 256: a row's weight is its probability times its scale, so a row of large values and no probability
//    takes nothing from the others.  P' = hi - lo with hi in e4m3 and lo in e5m2, each to nearest: off by
//    2^-8 of itself, as bf16 would be, from 2^-6 on (hi has four bits, lo three of the rest), and by 2^-13
//    below (hi is a multiple of 2^-9): 2^-17 of the head's largest p 2^e.  O^T += C^T (hi - lo), d = 512
//    as four blocks of 128 lanes, heads as columns; l = sum of P' 2^-e_r of the unrounded f32 P', which is
//    2^(4 - m) times the denominator, so O 2^-12 / (l + 2^(sink + 4 - m)) is the output.  P' below 2^-126 is 0: a
//    row D octaves below the one that sets m loses its part in l from 2^(D - 130) of that one's probability on.
//
// Why so.  A tile is 128 rows of 512 bytes, so two tiles, q (64 KB as hi and lo) and P fit the 227 KB of an
// SM; as bf16 only tiles of 64 rows would, and a 64-row tcgen05.mma takes the time of a 128-row one.  With
// N = 128 in S and K = 32 a step a tile takes 16 + 32 instructions where bf16 rows would take 64 + 64.  The price is
// q and P in two 8-bit pieces each, which is a choice: with one piece each would keep four bits; a third for P
// would add half to P V's instructions, and to the conversions, for bits that the output, bf16, mostly drops
// (errors against 64 bits: 0.0018-0.0020 of the output, 0.0017 with everything in f32 before its rounding).  The
// widening to e5m2 goes through f16: a conversion and a product for two codes, a byte permute for four.
//
// Warps: 0-7 softmax and epilogue (warp w: TMEM lanes 32 (w % 4).., heads 32 (w / 4)..), 8-15 rows (codes
// loaded a tile ahead into registers, widened into the swizzled stage; q at a unit's first tile), 16 MMA
// issue, 17 index rows: it drops entries without a row, turns the others into row numbers and hands out tiles of
// up to 128 (a unit without rows gives one tile of none), 18-19 the exponents of a tile's rows, between
// the index warp and the row warps.  What a tile is (its rows, whether it is its unit's first or last) goes on
// with the stage.  The softmax holds 32 heads of scores a thread and the row warps eight row loads in flight, so
// of the launch's 96 registers a thread the softmax warps take 120 and leave the others 80; 16 softmax warps
// with half the heads, or 12 more row warps, were slower (more instructions in all, or spilled loads).  ptxas spills
// 36 bytes a thread.
// A unit is one token and up to 64 heads; units are shared out as in the other attention kernels
// (attn_split.cuh), and units cut by a range boundary leave f32 partials that a second kernel merges.
// Every wait is bounded (2 s): then DS_DEV_TIMEOUT is flagged, issued MMAs are drained, TMEM is freed.
//
// Measured (entries / heads): 256 tokens of 2176 / 128, 217 us (658 TFLOP/s; its MMAs alone 72 us);
// 4096 prefill tokens of up to 640 / 64, 523 us (523 TFLOP/s); 64 tokens of 128 / 64, 12.2 us; one token of 2176 / 16,
// 15.6 us.  No pipe is full (a scheduler issues 0.43 to 0.46 a cycle, tensor 18 to 31 %, ALU 33 to 38 %, DRAM 11 to 13 %):
// a stage is held from its widening (about 3000 cycles) through S (750, and 560 to its readers) and the softmax
// (3500) to the end of P V (1400 to 1900), and with two stages that chain of 9000 to 9700 sets most of the 5500
// cycles that a tile takes.  A unit's end (output, the next q) takes about 8500 more.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "attn_split.cuh"
#include "common.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "sparse_attn_fp4.cuh"

namespace dsattn {
namespace fp4 {

using namespace ptx;
using split::kMaxCut;
using split::range_start;

constexpr int D = 512;
constexpr int HM = 64;                  // heads of a unit
constexpr int BN = 128;                 // rows of a tile
constexpr int NPAN = D / 128;           // panels of 128 columns
constexpr int PANEL = BN * 128;         // bytes of a panel: 128 rows (of C or of [hi | lo]) of 128
constexpr int STAGE = NPAN * PANEL;     // 64 KB
constexpr int NR = 4;                   // index messages
constexpr int NSOFTW = 8, NSOFT = 32 * NSOFTW, HPW = 32;    // softmax warps; heads of one
constexpr int W_ROWS = NSOFTW, NROWW = 8, W_MMA = W_ROWS + NROWW, W_IDX = W_MMA + 1, W_EXP = W_IDX + 1, NTHREADS = 640;
// Of eight heads of a range's first q a row warp takes this many and a softmax warp, idle until then, the others
// (64 tokens of 128 entries: 12.1 us; with three 12.35, with four half a microsecond more)
constexpr int QROWS = 2;
constexpr int RPL = BN / (2 * NROWW);                // steps of two rows that a row warp takes a tile
// of the 96 registers a thread of the launch the softmax warps take more (see above)
constexpr uint32_t REG_SOFT = 120, REG_OTHER = 80;
static_assert(NSOFT * REG_SOFT + (NTHREADS - NSOFT) * REG_OTHER <= NTHREADS * 96, "register split");
constexpr int SM_Q = 0;
constexpr int SM_KV = SM_Q + STAGE;
constexpr int SM_P = SM_KV + 2 * STAGE;
constexpr int P_BYTES = BN * 128;       // row r: 64 bytes hi, 64 bytes lo
constexpr int SM_CTL = SM_P + P_BYTES;
// control block
constexpr int C_ROWS = 0;                       // [NR][128] int32 row numbers
constexpr int C_EXPS = C_ROWS + NR * BN * 4;    // [NR][128][16] k - e_r + 27 of the rows' blocks (0: out of reach)
constexpr int C_TOPS = C_EXPS + NR * BN * (D / 32);   // [NR][128] int8 e_r
constexpr int C_REXP = C_TOPS + NR * BN;        // [2][128] int8 e_r of the stages' rows
constexpr int C_MAX = C_REXP + 2 * BN;          // [4][64] f32 maxima of the quarters
constexpr int C_SUM = C_MAX + 4 * HM * 4;       // [4][64] f32 sums of the quarters, at a unit's end
constexpr int C_HEAD = C_SUM + 4 * HM * 4;      // [64] f32 minus the running maximum m, 0 at a unit's start
constexpr int C_FAC = C_HEAD + HM * 4;          // [64] f32 factor of O^T: at m's rise, and at a unit's end
constexpr int C_QS = C_FAC + HM * 4;           // [2][64] f32 2^g scale log2(e), by unit parity
constexpr int C_BAR = C_QS + 2 * HM * 4;
enum : int {
    B_MSG = 0,                  // [NR] index -> exponents: message written
    B_EXP = B_MSG + NR,         // [NR] exponents -> rows: message and exponents written
    B_MSGFREE = B_EXP + NR,     // [NR] rows -> index
    B_KV = B_MSGFREE + NR,      // [2] rows -> MMA, softmax: stage and its meta written (and q, at a unit's first tile)
    B_PV = B_KV + 2,            // [2][2] MMA -> rows, softmax: P V of the tile's rows 64 k .. done
    B_S = B_PV + 4,             // [2] MMA -> softmax, rows: scores ready
    B_SFREE = B_S + 2,          // [2] softmax -> MMA: scores read
    B_P = B_SFREE + 2,          // softmax -> MMA: P written
    B_Q = B_P + 1,              // softmax -> MMA: their share of the first q written
    B_DRAIN = B_Q + 1,
    B_COUNT = B_DRAIN + 1
};
constexpr int C_MSG = C_BAR + 8 * B_COUNT;      // [NR] int32 message heads
constexpr int C_META = C_MSG + 4 * NR;          // [2] int32 the stages' messages
constexpr int C_TMEM = C_META + 8;
constexpr int C_ABORT = C_TMEM + 4;
constexpr int SMEM_BYTES = SM_CTL + C_ABORT + 4;
static_assert(C_BAR % 8 == 0 && SMEM_BYTES <= 232448, "shared memory budget");

constexpr int TM_O = 0, TM_S = NPAN * HM, TMEM_COLS = 512;
static_assert(TM_S + 2 * 2 * HM <= TMEM_COLS, "TMEM budget");

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTop = 4;                 // octaves of P' at m
constexpr int kMinExp = -96, kMaxExp = 100;     // of e_r
constexpr float kSlack = 4.0f;          // octaves that m may be late
constexpr uint32_t kAll = 0xffffffffu;

// messages: kind | first tile of its unit << 8 | last << 9 | the unit is whole << 10 | the range's first << 11 |
// the unit is padding << 12 | rows << 16
constexpr int kTile = 1, kFin = 2, kFirst = 1 << 8, kLast = 1 << 9, kWhole = 1 << 10, kSlot0 = 1 << 11, kPad = 1 << 12;

// a partial slot (f32): O [64][512], then running maxima m [64] (octaves, -inf: no row) and sums l [64]
constexpr int SLOT_O = HM * D;
constexpr size_t SLOT = (size_t)SLOT_O + 2 * HM;

struct Params {
    Args a;
    int ntok, nunit;
    int groups;       // units of a token
    int G;
    int seg_cost;
    bool interleave;
    float scale_log2;
    float *ws;
    int stall_first_tile;
};

__host__ __device__ constexpr uint32_t idesc8(int M, int N, int afmt, int bfmt, bool mn, bool minus = false) {
    // kind::f8f6f4: f32 accumulator; formats 0 = e4m3, 1 = e5m2; both operands K-major or MN-major; B negated
    return (1u << 4) | ((uint32_t)afmt << 7) | ((uint32_t)bfmt << 10) | ((minus ? 1u : 0u) << 14) | ((mn ? 3u : 0u) << 15) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of a converged warp.  Behind it (and not behind lane == 0) the compiler keeps what is the same for the
// warp in uniform registers, where the MMA's operands have to be: 5 instructions an MMA instead of 15.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// NaN where any value is one (warp_max leaves them out)
__device__ __forceinline__ float warp_max_nan(float v) {
    float r;
    asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ bool bar_or(bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(pred ? 1u : 0u), "n"(NSOFT)
        : "memory");
    return r != 0;
}

// One try at a phase that lets the hardware suspend the thread for up to NS nanoseconds.
template <int NS>
__device__ __forceinline__ bool try_hint(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(NS)
        : "memory");
    return ok != 0;
}

// Bounded wait of a whole warp; false when it gave up, or another role did.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort) {
    uint64_t t0 = 0;
    while (!__all_sync(kAll, try_hint<20000>(bar, parity))) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) *abort = 1;
        if (__any_sync(kAll, *abort != 0)) return false;
    }
    return true;
}

// 2^k, 0 below the normal numbers
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)max(k + 127, 0) << 23); }

__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t s) { return __byte_perm(a, b, s); }

// two f32 to e4m3, lo in the low byte; nearest, saturating
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
// A pair of bf16 values times f (a power of two, as a bf16 pair; their products are below 256) as hi + 2^-5 lo, both
// e4m3 to nearest.  As f16 the products are exact, but for multiples of 2^-24 below 2^-17.
__device__ __forceinline__ void split_q(uint32_t w, uint32_t f, uint32_t &hi, uint32_t &lo) {
    uint16_t h, l;
    asm("{\n\t.reg .b32 y, a, b, x, r;\n\t"
        "mul.rn.bf16x2 y, %2, %3;\n\t"
        "shl.b32 a, y, 16;\n\t"
        "and.b32 b, y, 0xffff0000;\n\t"
        "cvt.rn.f16x2.f32 x, b, a;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %0, x;\n\t"
        "cvt.rn.f16x2.e4m3x2 r, %0;\n\t"
        "sub.rn.f16x2 r, x, r;\n\t"
        "mul.rn.f16x2 r, r, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 %1, r;\n\t}"
        : "=&h"(h), "=&h"(l)
        : "r"(w), "r"(f), "r"(0x50005000u));     // 32, twice
    hi = h;
    lo = l;
}

// 16 bytes of the cache that no L1 line is kept for: beside 220 KB of shared memory L1 has 28 KB, less than the
// rows of a tile in flight.
__device__ __forceinline__ uint4 ld_row(const void *ptr) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(ptr));
    return v;
}

// One head of q (16 values a lane; sign: its sign bit is flipped) into [hi | lo]; returns g.  Where a value is not
// finite, all of the head's hi are NaN (e4m3 has no infinity to hand one on).
__device__ __forceinline__ int put_q(uint32_t sq, int hh, const uint4 (&v)[2], int lane, uint32_t sign) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t top2 = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top2 = __vmaxu2(top2, w[k] & 0x7fff7fffu);
    const uint32_t top = __reduce_max_sync(kAll, max(top2 & 0xffffu, top2 >> 16));
    const int g = max((int)(top >> 7) - 127 - 7, -126);      // the largest value lies in [128, 256) 2^g
    const uint32_t down = (((uint32_t)(127 - g) << 7) | sign) * 0x10001u;
    const uint32_t nan = top >= 0x7f80u ? 0x7f7fu : 0u;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t h2, l2;
        split_q(w[k], down, h2, l2);
        h2 |= nan;
        hi[k >> 1] = k & 1 ? hi[k >> 1] | (h2 << 16) : h2;
        lo[k >> 1] = k & 1 ? lo[k >> 1] | (l2 << 16) : l2;
    }
    const uint32_t at = sq + (uint32_t)(lane >> 3) * PANEL + (uint32_t)hh * 128 + (uint32_t)(((lane & 7) ^ (hh & 7)) * 16);
    st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
    st_shared_v4(at + HM * 128, lo[0], lo[1], lo[2], lo[3]);
    return g;
}

// Token of a position in the token order (split::unit_at; the launch keeps the numbers below 2^31).
__device__ __forceinline__ int token_at(uint32_t i, int ntok, bool interleave) {
    return interleave ? (i & 1u ? ntok - 1 - (int)(i >> 1) : (int)(i >> 1)) : (int)i;
}

// Unit of a position in the unit order: groups of a token are neighbours, so that their gathers meet in L2.
struct Unit {
    int tok, h0, nh;
};
__device__ __forceinline__ Unit unit_of(const Params &p, uint32_t u) {
    const int g = p.groups == 1 ? 0 : (int)(u & 1u);
    return {token_at(p.groups == 1 ? u : u >> 1, p.ntok, p.interleave), g * HM, min(HM, p.a.h - g * HM)};
}

// Heads hh .. hh + n - 1 of a unit's q into [hi | lo], the next two heads in flight; lane i < n gets the scale of head
// hh + i, 2^g |scale| log2(e).  ready(), between the first loads and the first store, says whether to go on.
template <typename F>
__device__ __forceinline__ float put_heads(const Params &p, uint32_t sq, uint32_t unit, int hh, int n, int lane, F ready) {
    const Unit un = unit_of(p, unit);
    const uint4 *src = reinterpret_cast<const uint4 *>(p.a.q + ((int64_t)un.tok * p.a.h + un.h0 + hh) * D) + 2 * lane;
    const uint32_t sign = p.scale_log2 < 0.0f ? 0x8000u : 0u;
    const int there = min(un.nh - hh, n);
    uint4 v[3][2];
    auto load = [&](uint4 (&to)[2], int i) {
        to[0] = to[1] = make_uint4(0, 0, 0, 0);
        if (i < there) {
            to[0] = __ldg(src + i * (D / 8));
            to[1] = __ldg(src + i * (D / 8) + 1);
        }
    };
    load(v[0], 0);
    load(v[1], 1);
    float qs = 0.0f;
    if (!ready()) return qs;
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        load(v[2], i + 2);
        const int g = put_q(sq, hh + i, v[0], lane, sign);
        if (lane == i) qs = fabsf(p.scale_log2) * pow2(g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            v[0][k] = v[1][k];
            v[1][k] = v[2][k];
        }
    }
    return qs;
}

// The 32 codes of a block at 2^(y - 15) in e5m2: pairs widened to f16, times the f16 number whose exponent field
// is y (exact; y = 0 is zero), and the high bytes of the f16 values, which are e5m2 (e2m1 has one
// mantissa bit, e5m2 two).
__device__ __forceinline__ void widen(const uint4 raw, uint32_t y, uint32_t (&o)[8]) {
    const uint32_t sc = y * 0x04000400u;
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t.reg .b32 f0, f1, f2, f3;\n\t"
            "mov.b32 {c0, c1, c2, c3}, %2;\n\t"
            "cvt.rn.f16x2.e2m1x2 f0, c0;\n\t"
            "cvt.rn.f16x2.e2m1x2 f1, c1;\n\t"
            "cvt.rn.f16x2.e2m1x2 f2, c2;\n\t"
            "cvt.rn.f16x2.e2m1x2 f3, c3;\n\t"
            "mul.rn.f16x2 f0, f0, %3;\n\t"
            "mul.rn.f16x2 f1, f1, %3;\n\t"
            "mul.rn.f16x2 f2, f2, %3;\n\t"
            "mul.rn.f16x2 f3, f3, %3;\n\t"
            "prmt.b32 %0, f0, f1, 0x7531;\n\t"
            "prmt.b32 %1, f2, f3, 0x7531;\n\t}"
            : "=r"(o[2 * k]), "=r"(o[2 * k + 1])
            : "r"(w[k]), "r"(sc));
}

// Four bytes of max(k, low) - low (signed k and low, biased to unsigned so that no byte borrows).
__device__ __forceinline__ uint32_t above(uint32_t k, uint32_t low) {
    return (__vmaxs4(k, low) ^ 0x80808080u) - (low ^ 0x80808080u);
}

// Four probabilities as hi (e4m3) - lo (e5m2): lo from hi - p, which is exact in f32.
__device__ __forceinline__ void split_p(uint64_t p01, uint64_t p23, uint32_t &hi, uint32_t &lo) {
    asm("{\n\t.reg .b32 f, g;\n\t.reg .b16 h0, h1, l0, l1, f0, f1, g0, g1;\n\t.reg .f32 p0, p1, p2, p3;\n\t"
        "mov.b64 {p0, p1}, %2;\n\t"
        "mov.b64 {p2, p3}, %3;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h0, p1, p0;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h1, p3, p2;\n\t"
        "cvt.rn.f16x2.e4m3x2 f, h0;\n\t"
        "cvt.rn.f16x2.e4m3x2 g, h1;\n\t"
        "mov.b32 {f0, f1}, f;\n\t"
        "mov.b32 {g0, g1}, g;\n\t"
        "sub.rn.f32.f16 p0, f0, p0;\n\t"
        "sub.rn.f32.f16 p1, f1, p1;\n\t"
        "sub.rn.f32.f16 p2, g0, p2;\n\t"
        "sub.rn.f32.f16 p3, g1, p3;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 l0, p1, p0;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 l1, p3, p2;\n\t"
        "mov.b32 %0, {h0, h1};\n\t"
        "mov.b32 %1, {l0, l1};\n\t}"
        : "=r"(hi), "=r"(lo)
        : "l"(p01), "l"(p23));
}

// One step of summing 32 values over a warp: lanes O apart share the first 2 O of them out.
template <int O>
__device__ __forceinline__ void fold(float (&l)[HPW], int lane) {
    const bool up = (lane & O) != 0;
#pragma unroll
    for (int i = 0; i < O; ++i) {
        const float give = up ? l[i] : l[i + O];
        l[i] = (up ? l[i + O] : l[i]) + __shfl_xor_sync(kAll, give, O);
    }
}

// 16 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

// whether a token lies behind its sequence's last one: nothing is read for it (but its q) or written
__device__ __forceinline__ bool is_padding(const Args &a, int tok) {
    if (!a.lens) return false;
    const uint32_t bi = (uint32_t)tok / (uint32_t)a.m;
    return tok - (int)bi * a.m >= __ldg(a.lens + bi);
}

// sin and cos of the output's rotation back, or null
__device__ __forceinline__ const float2 *rotation_row(const Args &a, int tok, bool flag) {
    const uint32_t bi = (uint32_t)tok / (uint32_t)a.m;
    const int64_t pos = (int64_t)__ldg(a.first + bi) + (tok - (int)bi * a.m);
    if (pos < 0 || pos >= a.table_rows) {
        if (flag) flag_status(a.status, DS_DEV_BAD_INDEX);
        return nullptr;
    }
    return a.table + pos * (a.rd / 2);
}

// S^T of a tile: rows of the stage by [hi | lo], 32 columns (bytes) a step.
template <uint32_t IDESC>
__device__ __forceinline__ void issue_s(uint32_t rows, uint32_t q, uint32_t d) {
    const uint64_t a = smem_desc_sw128(rows, 16, 1024), b = smem_desc_sw128(q, 16, 1024);
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
        const uint64_t off = (uint64_t)(((k >> 2) * PANEL + (k & 3) * 32) >> 4);
        mma_f8(d, a + off, b + off, IDESC, k ? 1u : 0u);
    }
}

// Half of O^T += C^T P, two steps of 32 rows: panel c's 128 columns as M (one 128-byte atom), a step's rows as K (four
// groups of eight, 1024 bytes apart); P the same with its 64 heads as N, hi then lo.
template <uint32_t I_HI, uint32_t I_LO>
__device__ __forceinline__ void issue_pv(uint32_t rows, uint32_t pr, uint32_t d, uint32_t keep) {
    const uint64_t a = smem_desc_sw128(rows, PANEL, 1024), b = smem_desc_sw128(pr, P_BYTES, 1024);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int c = 0; c < NPAN; ++c) {
            const uint64_t ao = a + (uint64_t)((c * PANEL + k * 4096) >> 4), bo = b + (uint64_t)((k * 4096) >> 4);
            mma_f8(d + c * HM, ao, bo, I_HI, k ? 1u : keep);
            mma_f8(d + c * HM, ao, bo + (64 >> 4), I_LO, 1u);
        }
    }
}

template <bool ROPE>
__global__ void __launch_bounds__(NTHREADS, 1) sparse_attn_fp4_kernel(const Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    uint8_t *ctl = smem + SM_CTL;
    auto BAR = [&](int i) -> uint32_t { return base + SM_CTL + C_BAR + 8u * (uint32_t)i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(ctl + C_ABORT);
    const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int T = p.a.topk;
    const int64_t cid = blockIdx.x;
    const int64_t e0 = range_start(cid, p.nunit, T, p.seg_cost, p.G);
    const int64_t e1 = range_start(cid + 1, p.nunit, T, p.seg_cost, p.G);
    const uint32_t u0 = (uint32_t)(e0 / T);

    if (threadIdx.x == 0) {
        for (int i = 0; i < NR; ++i) {
            mbar_init(BAR(B_MSG + i), 1);
            mbar_init(BAR(B_EXP + i), 2);
            mbar_init(BAR(B_MSGFREE + i), NROWW);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(B_KV + i), NROWW);
            for (int k = 0; k < 2; ++k) mbar_init(BAR(B_PV + 2 * i + k), 1);
            mbar_init(BAR(B_S + i), 1);
            mbar_init(BAR(B_SFREE + i), NSOFTW);
        }
        mbar_init(BAR(B_P), NSOFTW);
        mbar_init(BAR(B_Q), NSOFTW);
        mbar_init(BAR(B_DRAIN), 1);
        *abort_flag = (base & 1023u) != 0;       // the swizzled operands need this alignment
        fence_mbar_init();
        grid_launch_dependents();
    }
    if (warp == W_MMA) {
        tmem_alloc(base + SM_CTL + C_TMEM, TMEM_COLS);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kAll, *reinterpret_cast<volatile uint32_t *>(ctl + C_TMEM), 0);
    grid_dependency_wait();
    volatile int *msgs = reinterpret_cast<volatile int *>(ctl + C_MSG);

    volatile int *meta = reinterpret_cast<volatile int *>(ctl + C_META);
    if (warp >= W_ROWS) setmaxnreg_dec<REG_OTHER>();

    if (warp == W_IDX) {
        // ================================ index rows to tiles of row numbers ================================
        uint32_t n = 0;
        auto open = [&]() -> bool {               // the slot of message n is free
            return n < NR || warp_wait(BAR(B_MSGFREE + n % NR), (n / NR - 1) & 1u, abort_flag);
        };
        auto publish = [&](int msg) {
            if (lane == 0) msgs[n % NR] = msg;
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_MSG + n % NR));
            ++n;
        };
        bool ok = true, flagged = false;
        for (uint32_t u = u0; ok && (int64_t)u * T < e1; ++u) {
            const Unit un = unit_of(p, u);
            const int32_t *idx = p.a.idx + (int64_t)un.tok * T;
            const int32_t *bt = p.a.block_table + (int64_t)((uint32_t)un.tok / (uint32_t)p.a.m) * p.a.max_pages;
            const int a = u == u0 ? (int)(e0 - (int64_t)u * T) : 0;
            int z = (int)min((int64_t)T, e1 - (int64_t)u * T);
            int tile = kTile | (a == 0 && z == T ? kWhole : 0) | (u == u0 ? kSlot0 : 0);
            if (is_padding(p.a, un.tok)) {      // one tile of no rows, whose output is not written
                z = a;
                tile |= kPad;
            }
            int fill = 0, first = kFirst;
            int nxt[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) nxt[k] = a + 32 * k + lane < z ? __ldg(idx + a + 32 * k + lane) : -1;
            ok = open();
            int32_t *slot = reinterpret_cast<int32_t *>(ctl + C_ROWS) + (n % NR) * BN;
            for (int j = a; ok && j < z; j += 128) {
                int row[4], pg[4];
                bool bad = false;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t r = (uint32_t)nxt[k];
                    const uint32_t q = r / (uint32_t)p.a.page;
                    row[k] = nxt[k] < 0 ? -1 : (int)(r - q * (uint32_t)p.a.page);
                    pg[k] = nxt[k] < 0 ? 0 : q < (uint32_t)p.a.max_pages ? __ldg(bt + q) : -1;
                    const int jj = j + 128 + 32 * k + lane;
                    nxt[k] = jj < z ? __ldg(idx + jj) : -1;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (row[k] >= 0) {
                        if (pg[k] < 0 || pg[k] >= p.a.pages) {
                            bad = true;
                            row[k] = -1;
                        } else {
                            row[k] += pg[k] * p.a.page;
                        }
                    }
                    const uint32_t have = __ballot_sync(kAll, row[k] >= 0);
                    const int at = fill + __popc(have & lanemask_lt());
                    if (row[k] >= 0 && at < BN) slot[at] = row[k];
                    fill += __popc(have);
                    if (fill > BN) {     // a full tile goes out once it is known not to be the last
                        publish(tile | first | (BN << 16));
                        first = 0;
                        ok = ok && open();
                        slot = reinterpret_cast<int32_t *>(ctl + C_ROWS) + (n % NR) * BN;
                        if (ok && row[k] >= 0 && at >= BN) slot[at - BN] = row[k];
                        fill -= BN;
                    }
                }
                if (bad && !flagged) {
                    flag_status(p.a.status, DS_DEV_BAD_INDEX);
                    flagged = true;
                }
            }
            if (ok) publish(tile | first | kLast | (fill << 16));
        }
        if (ok && open()) publish(kFin);
    } else if (warp >= W_ROWS && warp < W_MMA) {
        // ======================== rows (and q) into the swizzled operands ========================
        // Warp w takes rows 4 w .. 4 w + 3 of each 32 (of each step of P V), two a step: step i rows
        // 32 (i / 2) + 4 w + 2 (i % 2) + 0, 1.  Lane: panel lane / 8, row (lane / 4) % 2 of the two, block lane % 4
        // of the panel.  Eight neighbouring lanes then store to all eight 16-byte columns of a 128-byte row:
        // the even ones from the even row, the odd ones from the odd row.
        const int w = warp - W_ROWS, panel = lane >> 3, half = (lane >> 2) & 1, u = panel * 4 + (lane & 3);
        uint32_t at[2];                                      // of the block's first half in step i % 2
#pragma unroll
        for (int i = 0; i < 2; ++i)
            at[i] = base + SM_KV + (uint32_t)panel * PANEL + (uint32_t)(4 * w + 2 * i + half) * 128 +
                    (uint32_t)(((lane & 3) * 2 ^ (4 * (w & 1) + 2 * i + half)) * 16);
        uint32_t unit = u0;
        int msg = 0;
        uint32_t seg = 0;
        uint4 raw[RPL];                                      // codes of the tile in hand, 16 bytes a lane and step
        const uint8_t *codes = p.a.codes + u * 16;
        const int first_row = 4 * w + half;                  // of step 0
        auto next_msg = [&](uint32_t n) -> bool {
            if (!warp_wait(BAR(B_EXP + n % NR), (n / NR) & 1u, abort_flag)) return false;
            msg = msgs[n % NR];
            return true;
        };
        // step i of message n; a tile without rows loads nothing, its exponents are all 0
        auto load = [&](uint32_t n, int i) {
            const int r = reinterpret_cast<const int32_t *>(ctl + C_ROWS)[(n % NR) * BN + first_row + 32 * (i >> 1) + 2 * (i & 1)];
            if (msg >> 16) raw[i] = ld_row(codes + (int64_t)r * (D / 2));
        };
        bool ok = next_msg(0);
        if (ok) {
#pragma unroll
            for (int i = 0; i < RPL; ++i) {
                raw[i] = make_uint4(0, 0, 0, 0);
                load(0, i);
            }
        }
        for (uint32_t J = 0; ok; ++J) {
            const int tile = msg;
            const uint32_t st = J & 1u;
            if ((tile & 255) == kFin) {
                if (J >= 2 && !warp_wait(BAR(B_PV + 2 * st + 1), ((J >> 1) - 1) & 1u, abort_flag)) break;
                if (warp == W_ROWS && lane == 0) meta[st] = tile;
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_KV + st));
                break;
            }
            float qs = 0.0f;
            if (tile & kFirst) {
                // the unit's q, once S of the tile before has read the last one's; of the first, the softmax warps,
                // which have nothing else to do then, take a share
                qs = put_heads(p, base + SM_Q, unit, 8 * w, seg == 0 ? QROWS : 8, lane, [&]() -> bool {
                    return ok = J == 0 || warp_wait(BAR(B_S + (st ^ 1u)), ((J - 1) >> 1) & 1u, abort_flag);
                });
                if (!ok) break;
            }
            if (!next_msg(J + 1)) break;
            const uint8_t *exps = ctl + C_EXPS + ((J % NR) * BN + first_row) * (D / 32) + u;
#pragma unroll
            for (int i = 0; i < RPL; ++i) {
                // handed back by halves: each wait costs about as much as a step
                if (J >= 2 && (i & 3) == 0) ok = ok && warp_wait(BAR(B_PV + 2 * st + (i >> 2)), ((J >> 1) - 1) & 1u, abort_flag);
                uint32_t o[8];
                widen(raw[i], exps[(32 * (i >> 1) + 2 * (i & 1)) * (D / 32)], o);
                load(J + 1, i);                   // in flight until its turn
                const uint32_t to = at[i & 1] + st * STAGE + (uint32_t)(i >> 1) * 4096;
                st_shared_v4(to, o[0], o[1], o[2], o[3]);
                st_shared_v4(to ^ 16u, o[4], o[5], o[6], o[7]);
            }
            if (!ok) break;
            if (lane < 16)
                reinterpret_cast<int8_t *>(ctl + C_REXP)[st * BN + 16 * w + lane] =
                    reinterpret_cast<const int8_t *>(ctl + C_TOPS)[(J % NR) * BN + 16 * w + lane];
            if (warp == W_ROWS && lane == 0) meta[st] = tile;
            if (tile & kLast) ++unit;
            if (tile & kFirst) {
                // P V of tile J - 2 is done, so the softmax is through with the scales of two units ago
                if (lane < (seg == 0 ? QROWS : 8)) reinterpret_cast<float *>(ctl + C_QS)[((u0 + seg) & 1u) * HM + 8 * w + lane] = qs;
                ++seg;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(BAR(B_MSGFREE + J % NR));
                if (!(p.stall_first_tile && J == 0)) mbar_arrive(BAR(B_KV + st));
            }
        }
    } else if (warp >= W_EXP) {
        // ========================= exponents of the rows: lane = two rows =========================
        uint32_t unit = u0;
        for (uint32_t n = 0;; ++n) {
            if (!warp_wait(BAR(B_MSG + n % NR), (n / NR) & 1u, abort_flag)) break;
            const int msg = msgs[n % NR], count = (msg & 255) == kTile ? msg >> 16 : 0;
            int32_t *rows = reinterpret_cast<int32_t *>(ctl + C_ROWS) + (n % NR) * BN;
            const int r0 = count > 0 ? rows[0] : 0;
            uint4 ev[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = 64 * (warp - W_EXP) + 32 * k + lane;
                ev[k] = make_uint4(0, 0, 0, 0);
                if (i < count) ev[k] = ld_row(p.a.exps + (int64_t)rows[i] * (D / 32));
                else rows[i] = r0;                // beyond the count: the tile's first row, with exponents 0
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = 64 * (warp - W_EXP) + 32 * k + lane;
                const uint32_t m4 = __vmaxs4(__vmaxs4(ev[k].x, ev[k].y), __vmaxs4(ev[k].z, ev[k].w));
                int top = max(max((int)(int8_t)m4, (int)(int8_t)(m4 >> 8)), max((int)(int8_t)(m4 >> 16), (int)m4 >> 24));
                top = max(top, kMinExp);
                if (top > kMaxExp) {
                    constexpr uint32_t most = (uint32_t)kMaxExp * 0x01010101u;
                    ev[k] = make_uint4(__vmins4(ev[k].x, most), __vmins4(ev[k].y, most), __vmins4(ev[k].z, most),
                                       __vmins4(ev[k].w, most));
                    top = kMaxExp;
                    flag_status(p.a.status, DS_DEV_BAD_VALUE);
                }
                const uint32_t low = (uint32_t)(uint8_t)(top - 27) * 0x01010101u;
                const uint32_t on = i < count ? kAll : 0u;
                reinterpret_cast<uint4 *>(ctl + C_EXPS)[(n % NR) * BN + i] =
                    make_uint4(above(ev[k].x, low) & on, above(ev[k].y, low) & on, above(ev[k].z, low) & on,
                               above(ev[k].w, low) & on);
                reinterpret_cast<int8_t *>(ctl + C_TOPS)[(n % NR) * BN + i] = (int8_t)top;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_EXP + n % NR));
            if ((msg & 255) == kFin) break;
            // the q of the next unit on its way to L2: its loads wait for nothing else when their time comes
            if ((msg & kFirst) && (int64_t)++unit * T < e1) {
                const Unit un = unit_of(p, unit);
                const uint16_t *q = p.a.q + ((int64_t)un.tok * p.a.h + un.h0) * D;
                for (int i = 32 * (warp - W_EXP) + lane; i < un.nh * (D / 64); i += 64) prefetch_l2(q + i * 64);
            }
        }
    } else if (warp == W_MMA) {
        // ================================== MMA issue ==================================
        // The whole warp walks the loop (its conditions are votes), an elected lane issues.
        constexpr uint32_t I_S = idesc8(BN, 2 * HM, 1, 0, false);
        constexpr uint32_t I_HI = idesc8(128, HM, 1, 0, true), I_LO = idesc8(128, HM, 1, 1, true, true);
        auto done = [&](int bar, uint32_t phase) -> bool { return __all_sync(kAll, mbar_test_wait(BAR(bar), phase & 1u)); };
        uint32_t sJ = 0, vJ = 0, vk = 0;   // next tile of S and of P V, and its next half
        bool fin = false;                  // no more tiles
        uint32_t keep = 0;                 // bit J & 1: tile J adds to O^T (is not its unit's first)
        uint32_t idle = 0;
        uint64_t since = 0;
        while (!fin || vJ < sJ) {
            if (!fin && sJ - vJ < 2 && done(B_KV + (sJ & 1u), sJ >> 1) &&
                (sJ < 2 || done(B_SFREE + (sJ & 1u), (sJ >> 1) - 1)) && (sJ > 0 || done(B_Q, 0))) {
                const uint32_t st = sJ & 1u;
                const int msg = __shfl_sync(kAll, meta[st], 0);
                idle = 0;
                if ((msg & 255) == kFin) {
                    fin = true;
                    continue;
                }
                tc_fence_after();
                if (elect_one()) {
                    issue_s<I_S>(base + SM_KV + st * STAGE, base + SM_Q, tmem + TM_S + st * 2 * HM);
                    mma_commit(BAR(B_S + st));
                }
                __syncwarp();
                keep = (keep & ~(1u << st)) | ((msg & kFirst ? 0u : 1u) << st);
                ++sJ;
            } else if (vJ < sJ && (vk > 0 || done(B_P, vJ))) {
                // by halves, the rows of each handed back behind it: S of the next tile, for which the softmax waits,
                // goes in between when it can
                const uint32_t st = vJ & 1u;
                tc_fence_after();
                if (elect_one()) {
                    issue_pv<I_HI, I_LO>(base + SM_KV + st * STAGE + vk * 8192, base + SM_P + vk * 8192, tmem + TM_O,
                                         vk ? 1u : (keep >> st) & 1u);
                    mma_commit(BAR(B_PV + 2 * st + vk));
                }
                __syncwarp();
                vJ += vk;
                vk ^= 1u;
                idle = 0;
            } else {
                // nothing to issue: sleep on the likelier of the two for up to 100 ns
                if (vJ < sJ) try_hint<100>(BAR(B_P), vJ & 1u);
                else try_hint<100>(BAR(B_KV + (sJ & 1u)), (sJ >> 1) & 1u);
                if ((++idle & 63u) == 0u) {
                    const uint64_t now = globaltimer_ns();
                    if (idle == 64u) since = now;
                    else if (now - since > kWaitLimitNs) *abort_flag = 1;
                    if (__any_sync(kAll, *abort_flag != 0)) break;
                }
            }
        }
        if (__any_sync(kAll, *abort_flag != 0)) {   // let issued MMAs finish before TMEM is freed
            if (elect_one()) {
                mma_commit(BAR(B_DRAIN));
                mbar_wait_drain(BAR(B_DRAIN), 0, 100000000ull);
            }
        }
        __syncwarp();
    } else if (warp < NSOFTW) {
        // ============================ softmax and epilogue ============================
        setmaxnreg_inc<REG_SOFT>();
        // Warp (quarter, heads hb..): its 32 rows by its 32 heads of every tile, and in O^T its 32 lanes of every
        // panel by the same heads.  The four warps of the same heads agree on m without talking about it:
        // they read the same maxima.
        const int quarter = warp & 3, hb = (warp >> 2) * HPW, row = quarter * 32 + lane, hl = hb + lane;
        const uint32_t tm = tmem + ((uint32_t)(quarter * 32) << 16);
        float *head = reinterpret_cast<float *>(ctl + C_HEAD), *fac = reinterpret_cast<float *>(ctl + C_FAC), *sums = reinterpret_cast<float *>(ctl + C_SUM);
        const float *qs = reinterpret_cast<const float *>(ctl + C_QS);
        uint64_t l[HPW / 2];   // sums of P' 2^-e over this thread's rows, in pairs of heads
        float m = 0.0f;        // of head hl
        uint32_t unit = u0;
        bool bad = false;
        head[hl] = 0.0f;
        if (e0 < e1) {
            const float s = put_heads(p, base + SM_Q, unit, 8 * warp + QROWS, 8 - QROWS, lane, [] { return true; });
            if (lane < 8 - QROWS) const_cast<float *>(qs)[(u0 & 1u) * HM + 8 * warp + QROWS + lane] = s;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(B_Q));
        bar_or(false);
        for (uint32_t J = 0;; ++J) {
            const uint32_t st = J & 1u;
            bad = bad || *abort_flag || !warp_wait(BAR(B_KV + st), (J >> 1) & 1u, abort_flag);
            const int msg = bad ? 0 : meta[st];
            if ((msg & 255) == kFin) {
                if (bar_or(false)) bar_or(true);   // a warp that gave up meets the others here
                break;
            }
            // ---- a tile
            const int count = msg >> 16;
            const bool first = msg & kFirst;
            const bool live = row < count;
            float *maxima = reinterpret_cast<float *>(ctl + C_MAX);
            uint64_t v[HPW / 2];   // s + e - m + 4 in octaves, in pairs of heads
            int e = 0;
            bool late = true;      // m has to move
            if (!bad) bad = !warp_wait(BAR(B_S + st), (J >> 1) & 1u, abort_flag);
            if (!bad) {
                if (first) m = 0.0f;
                tc_fence_after();
                e = (int)reinterpret_cast<const int8_t *>(ctl + C_REXP)[st * BN + row];
                const float c = pow2(e - 12);
                const float e4 = (float)(e + kTop);
                const uint64_t cr = pair(c, c), low = pair(0.03125f, 0.03125f), er = pair(e4, e4);
                const float *q = qs + (unit & 1u) * HM + hb;
#pragma unroll
                for (int j = 0; j < HPW; j += 16) {
                    uint32_t r0[16], r1[16];
                    tmem_ld16(tm + TM_S + st * 2 * HM + hb + j, r0);
                    tmem_ld16(tm + TM_S + st * 2 * HM + HM + hb + j, r1);
                    tmem_wait16(r0);
                    tmem_wait16(r1);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 q4 = lds4(q + j + i), m4 = lds4(head + hb + j + i);
                        const uint64_t qv[2] = {pair(q4.x, q4.y), pair(q4.z, q4.w)}, mv[2] = {pair(m4.x, m4.y), pair(m4.z, m4.w)};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint64_t s = fma2(pair(__uint_as_float(r1[i + 2 * k]), __uint_as_float(r1[i + 2 * k + 1])), low,
                                                    pair(__uint_as_float(r0[i + 2 * k]), __uint_as_float(r0[i + 2 * k + 1])));
                            v[(j + i) / 2 + k] = add2(fma2(mul2(s, cr), qv[k], mv[k]), er);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(B_SFREE + st));
                if (!live) {       // a row beyond the tile's count
#pragma unroll
                    for (int i = 0; i < HPW / 2; ++i) v[i] = pair(-INFINITY, -INFINITY);
                }
                float top = -INFINITY;
#pragma unroll
                for (int i = 0; i < HPW / 2; ++i) {
                    float a, b;
                    unpair(v[i], a, b);
                    top = max3(top, a, b);
                }
                late = first || top > (float)kTop + kSlack;
            }
            if (bar_or(late)) {
                // the tile's maxima, and the heads' m behind them: always at a unit's first tile, seldom later
#pragma unroll
                for (int i = 0; i < HPW / 2; ++i) {
                    float a, b;
                    unpair(v[i], a, b);
                    a = warp_max(a);
                    b = warp_max(b);
                    if (lane == 0) *reinterpret_cast<float2 *>(maxima + quarter * HM + hb + 2 * i) = make_float2(a, b);
                }
                if (bar_or(bad)) break;
                const float t = fmaxf(fmaxf(maxima[hl], maxima[HM + hl]), fmaxf(maxima[2 * HM + hl], maxima[3 * HM + hl]));
                // up to the tile's maximum; no change when that is lower, or there is no row (-inf)
                const float up = first ? (t == -INFINITY ? 0.0f : t - kTop) : fmaxf(t - kTop, 0.0f);
                m += up;
                __syncwarp();
                head[hl] = -m;                         // the same from every quarter
                fac[hl] = ex2(-up);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < HPW / 2; ++i)
                    v[i] = add2(v[i], pair(-__shfl_sync(kAll, up, 2 * i), -__shfl_sync(kAll, up, 2 * i + 1)));
                if (first) {
#pragma unroll
                    for (int i = 0; i < HPW / 2; ++i) l[i] = 0;
                } else {
                    // this warp's part of O^T, and its sums, follow m
                    bad = !warp_wait(BAR(B_PV + 2 * (st ^ 1u) + 1), ((J - 1) >> 1) & 1u, abort_flag);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 2 * NPAN && !bad; ++c) {
                        const uint32_t at = tm + TM_O + (c >> 1) * HM + hb + (c & 1) * 16;
                        const float *f = fac + hb + (c & 1) * 16;
                        uint32_t r[16];
                        tmem_ld16(at, r);
                        tmem_wait16(r);
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f[i]);
                        tmem_st16(at, r);
                    }
                    tmem_st_wait();
#pragma unroll
                    for (int i = 0; i < HPW; i += 2) l[i / 2] = mul2(l[i / 2], pair(fac[hb + i], fac[hb + i + 1]));
                }
            }
            uint32_t hi[HPW / 4], lo[HPW / 4];
            {
                const float f = pow2(-e);
                const uint64_t fr = pair(f, f);
#pragma unroll
                for (int i = 0; i < HPW / 2; i += 2) {
                    uint64_t pr[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float a, b;
                        unpair(v[i + k], a, b);
                        pr[k] = pair(ex2(a), ex2(b));
                        l[i + k] = fma2(pr[k], fr, l[i + k]);
                    }
                    split_p(pr[0], pr[1], hi[i / 2], lo[i / 2]);
                }
            }
            // P is free once the tile before has been multiplied
            if (J > 0 && !bad) bad = !warp_wait(BAR(B_PV + 2 * (st ^ 1u) + 1), ((J - 1) >> 1) & 1u, abort_flag);
            const uint32_t pb = base + SM_P + (uint32_t)row * 128;
            const uint32_t c0 = (uint32_t)((hb >> 4) ^ (row & 7)) * 16;     // its 16-byte column; hb / 16 is even
            st_shared_v4(pb + c0, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(pb + (c0 ^ 16), hi[4], hi[5], hi[6], hi[7]);
            st_shared_v4(pb + (c0 ^ 64), lo[0], lo[1], lo[2], lo[3]);
            st_shared_v4(pb + (c0 ^ 80), lo[4], lo[5], lo[6], lo[7]);
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(B_P));
            if (msg & kLast) {
                // ---- the unit's output, or this range's part of it
                const bool whole = msg & kWhole;
                // sums over the warp's rows: lane i ends up with head hb + i
                float s[HPW];
#pragma unroll
                for (int i = 0; i < HPW; i += 2) unpair(l[i / 2], s[i], s[i + 1]);
                fold<16>(s, lane);
                fold<8>(s, lane);
                fold<4>(s, lane);
                fold<2>(s, lane);
                fold<1>(s, lane);
                sums[quarter * HM + hl] = s[0];
                const Unit un = unit_of(p, unit);
                ++unit;
                // what the output needs from memory, fetched while P V of the last tile runs
                float sink = 0.0f;
                const float2 *cs = nullptr;
                if (whole && !(msg & kPad)) {
                    if (hl < un.nh) sink = __ldg(p.a.sink + un.h0 + hl) * kLog2e;
                    if constexpr (ROPE) cs = rotation_row(p.a, un.tok, threadIdx.x == 0);
                }
                bad = bad || !warp_wait(BAR(B_PV + 2 * st + 1), (J >> 1) & 1u, abort_flag);
                tc_fence_after();
                if (bar_or(bad)) break;
                float *ws = p.ws + ((size_t)cid * 2 + (msg & kSlot0 ? 0 : 1)) * SLOT;
                const float sum = sums[hl] + sums[HM + hl] + sums[2 * HM + hl] + sums[3 * HM + hl];
                const bool any = sum != 0.0f;              // false: no rows (NaN counts)
                float f = 0x1p-12f;                        // of head hl
                if (whole) {
                    f = any ? 0x1p-12f / (sum + exp2f(sink - m + kTop)) : 0.0f;
                } else if (quarter == 0) {
                    ws[SLOT_O + hl] = any ? m : -INFINITY;
                    ws[SLOT_O + HM + hl] = sum;
                }
                __syncwarp();
                fac[hl] = f;                               // the same from every quarter
                head[hl] = 0.0f;
                __syncwarp();
#pragma unroll 1
                for (int k = msg & kPad ? 2 * NPAN : 0; k < 2 * NPAN; ++k) {
                    const int c = k >> 1, h0 = hb + (k & 1) * 16, d = c * 128 + row;
                    if (h0 >= un.nh) continue;
                    uint32_t r[16];
                    float x[16];
                    tmem_ld16(tm + TM_O + c * HM + h0, r);
                    tmem_wait16(r);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 f4 = lds4(fac + h0 + i);
                        unpair(mul2(pair(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), pair(f4.x, f4.y)), x[i], x[i + 1]);
                        unpair(mul2(pair(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])), pair(f4.z, f4.w)), x[i + 2],
                               x[i + 3]);
                    }
                    if (whole) {
                        // neighbouring lanes trade, so that each stores a pair of columns: the even one of head i, the
                        // odd one of head i + 1
                        const bool odd = lane & 1;
                        uint32_t *col = reinterpret_cast<uint32_t *>(
                            p.a.o + ((int64_t)un.tok * p.a.h + un.h0 + h0) * D + d + (odd ? D - 1 : 0));
                        uint32_t w[8];
                        if (ROPE && cs && c * 128 + quarter * 32 + 31 >= D - p.a.rd) {
                            float2 t = make_float2(1.0f, 0.0f);
                            if (d >= D - p.a.rd) t = __ldg(cs + ((d - (D - p.a.rd)) >> 1));
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float y = __shfl_xor_sync(kAll, odd ? x[2 * i] : x[2 * i + 1], 1);
                                const float lo = odd ? y : x[2 * i], hi = odd ? x[2 * i + 1] : y;
                                w[i] = pack_bf16x2(lo * t.x + hi * t.y, hi * t.x - lo * t.y);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const uint32_t two = pack_bf16x2(x[2 * i], x[2 * i + 1]);     // the two heads
                                w[i] = prmt(two, __shfl_xor_sync(kAll, two, 1), odd ? 0x3276u : 0x5410u);
                            }
                        }
                        const int heads = un.nh - h0 - (odd ? 1 : 0);
                        if (heads >= 16) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) col[i * D] = w[i];
                        } else {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                if (2 * i < heads) col[i * D] = w[i];
                        }
                    } else {
                        float *col = ws + h0 * D + d;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (h0 + i < un.nh) col[i * D] = x[i];
                    }
                }
                tc_fence_before();
            }
        }
    }

    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) flag_status(p.a.status, DS_DEV_TIMEOUT);
    if (warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Merge the partials of the units that a range boundary cuts: block (cut unit, four heads), warp = head.  A lane
// has the first four parts' accumulators in flight before their weights are known.
// Bound by latency: against a thread for four columns of a head and one part after the other the whole call took
// 22.7 -> 21.9 us for 32 units in two parts, 222 -> 220 with 150 cut ones, 20.1 -> 19.5 for one in eight.
constexpr int kCombineHeads = 4;
struct CombineParams {
    Args a;
    int ntok;
    int groups;
    bool interleave;
    const float *ws;
    int parts;                    // of every unit, each in its range's first slot
};
struct CutParams : CombineParams {
    int4 cut[kMaxCut];            // {unit, first part, parts, slot bits}
};

// Which unit and parts a block merges: from the table, or block u's unit u in p.parts parts (a launch costs the host
// less without the table's 2.5 KB).
__device__ __forceinline__ int4 cut_of(const CombineParams &p, int i) { return make_int4(i, i * p.parts, p.parts, 0); }
__device__ __forceinline__ int4 cut_of(const CutParams &p, int i) { return p.cut[i]; }

template <bool ROPE, typename P>
__global__ void __launch_bounds__(32 * kCombineHeads) combine_kernel(const P p) {
    grid_dependency_wait();
    const int4 c = cut_of(p, blockIdx.x);
    const int tok = token_at((uint32_t)(p.groups == 1 ? c.x : c.x >> 1), p.ntok, p.interleave);
    const int h0 = p.groups == 1 ? 0 : (c.x & 1) * HM, hh = blockIdx.y * kCombineHeads + (threadIdx.x >> 5);
    if (hh >= HM || h0 + hh >= p.a.h || is_padding(p.a, tok)) return;
    auto part = [&](int i) { return p.ws + ((size_t)(c.y + i) * 2 + (((uint32_t)c.w >> i) & 1u)) * SLOT; };
    // lane i: statistics of part i (at most 32), and columns 128 j + 4 i .. of every part
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.0f;
    if (lane < c.z) {
        m = part(lane)[SLOT_O + hh];
        l = part(lane)[SLOT_O + HM + hh];
    }
    float4 x[4][4];
    auto load = [&](int i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (i + k >= c.z) break;
            const float4 *src = reinterpret_cast<const float4 *>(part(i + k) + hh * D) + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[k][j] = src[32 * j];
        }
    };
    load(0);
    const float top = warp_max_nan(m);
    float4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (top != -INFINITY) {
        const float w = m == -INFINITY ? 0.0f : exp2f(m - top);
        float den = w * l;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kAll, den, o);
        den += exp2f(__ldg(p.a.sink + h0 + hh) * kLog2e - top + kTop);
        const float inv = 1.0f / den;
        for (int i = 0;;) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (i + k >= c.z) break;
                const float wi = __shfl_sync(kAll, w, i + k);
                if (wi == 0.0f) continue;          // a part without rows has no accumulator
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[j].x += wi * x[k][j].x;
                    acc[j].y += wi * x[k][j].y;
                    acc[j].z += wi * x[k][j].z;
                    acc[j].w += wi * x[k][j].w;
                }
            }
            i += 4;
            if (i >= c.z) break;
            load(i);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv);
    }
    const float2 *cs = nullptr;
    if constexpr (ROPE) cs = rotation_row(p.a, tok, lane == 0 && hh == 0);
    uint16_t *o = p.a.o + ((int64_t)tok * p.a.h + h0 + hh) * D;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int d = 128 * j + 4 * lane;
        if (cs && d >= D - p.a.rd) {
            const float2 t0 = __ldg(cs + ((d - (D - p.a.rd)) >> 1)), t1 = __ldg(cs + ((d - (D - p.a.rd)) >> 1) + 1);
            acc[j] = make_float4(acc[j].x * t0.x + acc[j].y * t0.y, acc[j].y * t0.x - acc[j].x * t0.y,
                                 acc[j].z * t1.x + acc[j].w * t1.y, acc[j].w * t1.x - acc[j].z * t1.y);
        }
        *reinterpret_cast<uint2 *>(o + d) = make_uint2(pack_bf16x2(acc[j].x, acc[j].y), pack_bf16x2(acc[j].z, acc[j].w));
    }
}

__global__ void __launch_bounds__(256) none_kernel(const Args a) {
    const int tok = blockIdx.x;
    if (is_padding(a, tok)) return;
    uint4 *o = reinterpret_cast<uint4 *>(a.o + (int64_t)tok * a.h * D);
    for (int i = threadIdx.x; i < a.h * (D / 8); i += 256) o[i] = make_uint4(0, 0, 0, 0);
}

// ---- host side ---------------------------------------------------------------------------------------

constexpr int kMaxDev = 64;
int g_sms[kMaxDev];
std::atomic<int> g_test_stall{0};
std::mutex g_mutex;

// CTAs that run at once on a device, the current one (one per SM), 0 when the kernel cannot be configured.
int max_ctas(int dev) {
    if (dev < 0 || dev >= kMaxDev) return 0;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_sms[dev]) return g_sms[dev];
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    for (const void *k : {(const void *)sparse_attn_fp4_kernel<false>, (const void *)sparse_attn_fp4_kernel<true>})
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess) return 0;
    return g_sms[dev] = sms;
}

struct Plan {
    int64_t ntok, nunit, G, K;
    int groups;
    bool split;
    int ncut;
    int4 cut[kMaxCut];
};

// Fixed cost of a unit on the cost line (q, the epilogue), in index entries: two tiles' worth (256 tokens of 128
// heads and 2176 entries: 216 us; with one tile's worth 219, with one and a half 219; 4096 tokens of 640 entries:
// 519 either way).
constexpr int kSegCost = 2 * BN;

// The units (two a token at most) in 32 bits, an entry's place in its list with the two tiles that the index warp
// looks ahead in 31, and every place on the cost line in 64: at most 1023 ranges' worth of all the units' entries.
bool fits(int b, int m, int topk) {
    const int64_t ntok = (int64_t)b * m;
    return topk <= INT32_MAX - 2 * BN && ntok <= INT32_MAX / 2 && ntok <= (INT64_MAX >> 11) / ((int64_t)topk + kSegCost);
}

// Ranges for a problem.  With at least as many units as CTAs: one a CTA, cut where they fall.  With fewer, every unit
// gets k of them, the k of the least estimated time in tiles of 2.8 us: a unit's tiles one after the other (the second
// overlaps the first), and from two parts on the merge: its launch (2.4 us on the device, and with the workspace 6 us
// of the host's time, hence 1.3 tiles), the partials through L2, the parts in turn.
// Measured on the device, whole against parts of about one tile (64 heads): 1 token of 256 entries 13.8 us (14.4 in two),
// 384: 17.0 (14.5 in three), 1024: 16.4 in four, 15.3 in eight; 16 tokens of 1024: 17.3 in four, 18.2 in eight; 40
// tokens of 256: 14.0 (15.8 in two); 70 of 384: 17.5 (20.2 in two).  15 tokens of 356, 40 heads: 17.0 whole, 14.4 in
// three, but then 17 to 20 a call for the host.
int64_t ranges(int64_t nunit, int topk, int gmax) {
    if (nunit >= gmax) return gmax;
    const int64_t most = std::min<int64_t>({gmax / nunit, ((int64_t)topk + BN - 1) / BN, 32});
    int64_t best = 1;
    float least = INFINITY;
    for (int64_t k = 1; k <= most; ++k) {
        const int64_t part = (topk + k - 1) / k, tiles = (part + BN - 1) / BN;
        float cost = tiles <= 2 ? 0.6f * (float)(tiles - 1) : (float)tiles - 1.25f;
        if (k > 1) cost += 1.3f + (float)(nunit * k) / 120.0f + (float)k / 30.0f;
        if (cost < least) {
            least = cost;
            best = k;
        }
    }
    return nunit * best;
}

// The plan of a shape on the current device; each host thread keeps its last one (a decode loop asks for the
// same one for every layer and step).  Null when there is none.
const Plan *plan(int b, int m, int h, int topk) {
    thread_local Plan last;
    thread_local int key[5] = {-1, 0, 0, 0, 0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    if (key[0] == dev && key[1] == b && key[2] == m && key[3] == h && key[4] == topk) return &last;
    const int gmax = max_ctas(dev);
    if (gmax <= 0 || !fits(b, m, topk)) return nullptr;
    key[0] = -1;
    Plan &pl = last;
    pl.ntok = (int64_t)b * m;
    pl.groups = h > HM ? 2 : 1;
    pl.nunit = pl.ntok * pl.groups;
    pl.G = ranges(pl.nunit, topk, gmax);
    pl.K = split::seg_cost(pl.nunit, pl.G, kSegCost);
    pl.split = split::splits_units(pl.nunit, topk, pl.G, pl.K);
    pl.ncut = pl.split ? split::cut_units(pl.nunit, topk, pl.K, pl.G, pl.cut) : 0;
    const int k[5] = {dev, b, m, h, topk};
    for (int i = 0; i < 5; ++i) key[i] = k[i];
    return &last;
}

size_t workspace_bytes(const Plan &pl) { return pl.split ? (size_t)pl.G * 2 * SLOT * sizeof(float) : 0; }

}  // namespace fp4

void set_test_stall_fp4(bool on) { fp4::g_test_stall.store(on ? 1 : 0, std::memory_order_relaxed); }

bool sparse_attn_fp4_fits(int b, int m, int topk) { return fp4::fits(b, m, topk); }

size_t sparse_attn_fp4_workspace_bytes(int b, int m, int h, int topk) {
    if (topk == 0 || (int64_t)b * m == 0) return 0;
    const fp4::Plan *pl = fp4::plan(b, m, h, topk);
    return pl ? fp4::workspace_bytes(*pl) : 0;
}

int launch_sparse_attn_fp4_none(const fp4::Args &a, cudaStream_t stream) {
    fp4::none_kernel<<<(unsigned)(a.b * a.m), 256, 0, stream>>>(a);
    return launch_status();
}

int launch_sparse_attn_fp4(const fp4::Args &a, cudaStream_t stream) {
    const fp4::Plan *plan = fp4::plan(a.b, a.m, a.h, a.topk);
    if (!plan) return launch_failed();
    const fp4::Plan &pl = *plan;
    const size_t need = fp4::workspace_bytes(pl);
    if (a.workspace_bytes < need || (need && !a.workspace)) return DS_EWORKSPACE;
    if (pl.split && pl.ncut <= 0) return DS_EUNSUPPORTED;
    const bool rope = a.rd > 0, interleave = a.m > 1;
    fp4::Params p{a, (int)pl.ntok, (int)pl.nunit, pl.groups, (int)pl.G, (int)pl.K, interleave, a.scale * fp4::kLog2e,
                  static_cast<float *>(a.workspace), fp4::g_test_stall.load(std::memory_order_relaxed)};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.G, 1, 1);
    cfg.blockDim = dim3(fp4::NTHREADS, 1, 1);
    cfg.dynamicSmemBytes = fp4::SMEM_BYTES;
    cfg.stream = stream;
    // programmatic dependent launch: the set-up overlaps the previous kernel on the stream
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, rope ? fp4::sparse_attn_fp4_kernel<true> : fp4::sparse_attn_fp4_kernel<false>, p) !=
        cudaSuccess)
        return launch_failed();
    if (pl.split) {
        const fp4::CombineParams head{a, (int)pl.ntok, pl.groups, interleave, p.ws, (int)(pl.G / pl.nunit)};
        const int heads = a.h < fp4::HM ? a.h : fp4::HM;
        cfg.gridDim = dim3((unsigned)pl.ncut, (unsigned)((heads + fp4::kCombineHeads - 1) / fp4::kCombineHeads), 1);
        cfg.blockDim = dim3(32 * fp4::kCombineHeads, 1, 1);
        cfg.dynamicSmemBytes = 0;
        cudaError_t e;
        if (pl.G > pl.nunit) {
            e = cudaLaunchKernelEx(&cfg, rope ? fp4::combine_kernel<true, fp4::CombineParams> : fp4::combine_kernel<false, fp4::CombineParams>, head);
        } else {
            fp4::CutParams c;
            static_cast<fp4::CombineParams &>(c) = head;
            for (int i = 0; i < pl.ncut; ++i) c.cut[i] = pl.cut[i];
            e = cudaLaunchKernelEx(&cfg, rope ? fp4::combine_kernel<true, fp4::CutParams> : fp4::combine_kernel<false, fp4::CutParams>, c);
        }
        if (e != cudaSuccess) return launch_failed();
    }
    return DS_OK;
}

}  // namespace dsattn
