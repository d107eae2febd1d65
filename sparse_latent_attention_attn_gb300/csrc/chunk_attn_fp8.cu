// chunk_attn_fp8.cu -- attention of a chunk of new tokens over the paged cache of 8-bit rows.
//
// For the query (token t of sequence bi, head hh) at position p = first[bi] + t, over the rows that it sees (positions
// max(0, p - window + 1) .. p, and compressed rows 0 .. (p + 1) / ratio - 1):
//     s_j = scale q . k_j,  o = sum_j exp(s_j) k_j / (sum_j exp(s_j) + exp(sink[hh])),
// then the inverse rotation of the last rd values ("DeepSeek V4.1", attention/attend and attention/query-latent).
//
// Queries of neighbouring tokens see nearly the same rows, so a unit of work is up to 128 query rows (a sequence's
// tokens and heads in one line: any number of heads fills it) against the union of the rows that they see, window rows
// first and compressed rows behind them, in tiles of 128; each query's own range is a mask.  With rows of 512 values an
// accumulator of 128 queries in f32 fills the tensor memory of an SM, which leaves no room for scores.  So two SMs share
// a unit (a cluster of two CTAs, cta_group::2), each with 64 of its queries and with one half of d:
//   * S = Q K^T: M = 128 queries (64 a CTA), N = 128 rows (64 a CTA), K = 512.  A CTA's scores lie on all 128 lanes: query r
//     on lane r with rows 0-63 of the tile, and on lane r + 64 with rows 64-127.
//   * O^T += V^T P^T: M = 256 values of d (128 a CTA, twice), N = 128 queries (each CTA's P), K = 128 rows.  O^T takes 256
//     columns of tensor memory, and two tiles of scores 128.
// The tensor cores read both CTAs' operands, so no scores and no probabilities cross between the CTAs.  The MMAs of a tile
// take 0.75 + 0.53 us (23.3 ns for each of 32, 32.9 ns for each of 16, measured at 2070 MHz: 48 and 68 cycles, where 8192
// operations a cycle and SM would be 32 and 64, so 0.66 of that rate for S, 0.94 for P V, 0.78 for both).
//
// A code widens to bf16 exactly (at most four significant bits; its bits moved to a bf16's, times 2^(120 + k)).  Two forms:
//   * Sequences with one or two tiles of queries (decoding), or where the form below does not fit: each row is read once a tile, as codes, and widened in registers
//     on its way into shared memory, which spares a copy in HBM: 33/32 byte a value is all that is read.  Each CTA widens its
//     64 rows once, as K; for P V it needs its half of d of all 128, copied from K in the layout that it has: its own rows by
//     a warp, the other CTA's by the copy engine, 8 KB each (the engine with both takes 2 us a tile).  K is held until its
//     copies have been read, and V is filled when the last tile's P V is done, so the copies stand between two tiles: 3.3 us
//     a tile where the MMAs take 1.28.  (The rows passed through a ring in the workspace instead, V by TMA: 204 -> 241 us for
//     256 sequences of 2176 rows; V widened a second time by eight more warps: 252 -> 370.)
//   * Sequences with more (WIDE; prompts): several units read the same rows, so a kernel before widens them once, into the
//     workspace, and K and V come by TMA: 1.5 us a tile, and some 4 us between units, in which q is loaded and O^T read.
//     The host knows the block table's width, not how much of it is used: tables of more rows than the workspace may take
//     (plan()) are read in the other form (16 prompts' chunks of 512 tokens and 128 heads over 2176 rows: 3.1 ms with a table
//     of 2688 rows, 5.5 with one of 262272).
// An operand half is handed back as soon as its readers are done.
//
// (Times: calls captured in a graph, one behind the other, unless another kind is named.)
//
// The softmax works on a reference per query: kSlack octaves above the first tile's maximum, moved (by whole octaves, so that
// O^T and the sum are scaled exactly) only when a later maximum exceeds it.  So P is at most 1, as large as it may be beside
// rows near the end of bf16's range, and a number's distance from the maximum costs it nothing down to 2^-106 of that.  The
// reference is never more than 64 octaves below the sink, so that 1 / (sum + sink) is a normal number wherever an output is.
// P is rounded to bf16 for the product, as in ds_sparse_attn; the sum takes it unrounded.
//
// Few units are cut into parts of their rows, and so are those of a last round that would leave clusters without work; a
// kernel behind joins a unit's parts by their references and sums.
//
// Warps: 0-3 softmax; from 4 on output (and O^T's rescaling, on request): four, or eight with WIDE; 8-15 widen; one issues the
// MMAs (in the cluster's first CTA, for both); one fetches q by TMA; two have the halves of K copied to V, or bring K and V.
// What bounds the small calls is instructions: roles share their SM's issue slots and instruction caches, so a body that
// is twice as long costs other roles time too.  Every wait gives up after 2 s, or 60 s where it lasts as long as a unit
// (DS_DEV_TIMEOUT).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "chunk_attn_fp8.cuh"
#include "f32x2.cuh"
#include "ptx.cuh"
#include "row_norm.cuh"

namespace dsattn {
namespace chunk {

using namespace ptx;
using rows::Divisor;

constexpr int D = 512;
constexpr int BN = 128;                     // rows of a tile
constexpr int HR = 64;                      // of them widened for S by each CTA; also query rows of a CTA, at most
constexpr int W_OUT = 4;                    // warps 0-3 softmax, from 4 on output
// First warps of the roles.  WIDE: the rows come as bf16 from the workspace, by TMA; else as codes that eight warps widen.
template <bool WIDE>
struct Roles {
    static constexpr int kOut = WIDE ? 8 : 4;                            // output warps: one a lane quarter and block, or both blocks
    static constexpr int kWiden = 8, kMma = WIDE ? 12 : 16, kQ = kMma + 1, kCopy = 18, kLoad = 14;   // (two warps each: kCopy, kLoad)
    static constexpr int kThreads = WIDE ? 512 : 640;
};
// registers: 128 * (136 + 104 + 96 + 96 + 48) is what 640 threads have with 96 each
constexpr uint32_t REG_SOFTMAX = 136, REG_OUT = 104, REG_MMA = 48;

constexpr int K_CHUNK = HR * 128;           // 64 rows of 64 values
constexpr int V_CHUNK = BN * 128;           // 128 rows of 64 values
constexpr int SM_Q = 0;                     // 8 chunks of 64 query rows
constexpr int SM_K = SM_Q + 8 * K_CHUNK;    // 8 chunks
constexpr int SM_V = SM_K + 8 * K_CHUNK;    // 4 chunks (this CTA's half of d)
constexpr int P_BYTES = 2 * K_CHUNK;        // 64 query rows of 128 probabilities
constexpr int SM_P = SM_V + 4 * V_CHUNK;    // two buffers
constexpr int SM_CTL = SM_P + 2 * P_BYTES;
constexpr int SMEM_BYTES = SM_CTL + 3 * 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

constexpr int TM_O = 0, TM_S = 256, TM_COLS = 512;

// barriers (8 bytes each); "first": used in the cluster's first CTA only
enum : int {
    B_KFULL = 0,              // [2] half of K's chunks widened in both CTAs (first)
    B_KLOC = B_KFULL + 2,     // [2] ... in this CTA
    B_KFREE = B_KLOC + 2,     // [2] its MMAs are done, and its copies have been read
    B_VLOC = B_KFREE + 2,     // [2] half of V's chunks landed in this CTA
    B_VFULL = B_VLOC + 2,     // [2] ... in both (first)
    B_VFREE = B_VFULL + 2,    // [2] its MMAs are done
    B_S = B_VFREE + 2,        // [2] scores of tile J there (J & 1)
    B_P = B_S + 2,            // [2] P of tile J written in both CTAs (first)
    B_Q = B_P + 2,            // q of a unit landed in both CTAs (first)
    B_QFREE = B_Q + 1,        // the unit's last S is done
    B_O = B_QFREE + 1,        // for the output warps: the unit's last P V is done, or O^T is to be rescaled (C_EVENT)
    B_OFREE = B_O + 1,        // O^T read in both CTAs (first)
    B_INV = B_OFREE + 1,      // [2] the unit's factors (unit & 1) are there
    B_INVFREE = B_INV + 2,    // [2] both CTAs' output warps are done with them
    B_RESCD = B_INVFREE + 2,  // O^T rescaled in both CTAs (first)
    B_SYNC = B_RESCD + 1,     // P V so far is done (first)
    B_DRAIN = B_SYNC + 1,
    B_COUNT = B_DRAIN + 1
};
constexpr int C_TMEM = 8 * B_COUNT, C_ABORT = C_TMEM + 4, C_RESC = C_ABORT + 4;   // [2] int: tile + 1 that needs a rescale
constexpr int C_CNT = C_RESC + 8;                                                 // [4] int: tiles of the units under way
constexpr int C_EVENT = C_CNT + 16;         // [2] int: 2 (n + 1) + (J & 1) where phase n of B_O asks for a rescale at tile J
static_assert(C_EVENT + 8 <= 256, "control block");
constexpr int C_ALPHA = 256;                // [2][128] int16: octaves by which a query's column of O^T is to be lowered
constexpr int C_INV = C_ALPHA + 512;        // [2][128] f32: 1 / denominator
constexpr int C_XCH = C_INV + 1024;         // [2][2][64] f32: maxima and sums, between the two threads of a query
static_assert(SM_CTL + C_XCH + 1024 <= SMEM_BYTES, "control block");

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kUnitLimitNs = 30 * kWaitLimitNs;   // of waits that last as long as a unit
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 20.0f;             // octaves that a reference is put above the maximum
constexpr uint32_t kAll = 0xffffffffu;

struct Params {
    Args a;
    Divisor h, page, ring, b, parts, ratio;   // (a 64-bit division takes a warp half a microsecond, and every role makes its units)
    int R;               // query rows of a CTA: 64, 32 or 16
    int nqt;             // query tiles of a sequence
    uint32_t units;      // whole ones, then parts of the others
    uint32_t whole;
    Divisor clusters;
    int64_t cap;         // logical rows that the block table can hold, at most kMaxRows
    float scale_log2;
    float *ws;           // parts of units
    uint16_t *rows;      // WIDE: the sequences' rows in bf16, wrows of positions and crows compressed ones of each
    int wrows, crows;
    int stall;
};

// A unit's rows: tile t holds rows [128 t, 128 t + 128) of the list of nw window rows (positions wlo ..) and nc compressed
// rows, which begin at nwp >= nw; this unit takes tiles [t0, t1).  Logical rows are below kMaxRows, so what counts them fits an int.
constexpr int64_t kMaxRows = 1 << 29;
struct Unit {
    int bi, part;
    int r0, rows;        // query rows [r0, min(r0 + 2 R, rows)) of the sequence
    int first;
    uint32_t wlo;
    int nw, nwp, nc;
    int t0, t1;
    bool clipped;        // rows beyond the block table
};

// Which of a sequence's query tiles unit u is (of), of which sequence, and which part of it.  Later tokens see more, so
// the sequences' last tiles come first.  A cluster takes every `clusters`-th unit: the sequences change places
// from round to round (by a hash of the round), so that it does not get one sequence's units only.
struct Place {
    uint32_t of, bi, part;
    int qt;
};
__device__ __forceinline__ Place place_of(const Params &p, uint32_t of, uint32_t part) {
    Place x;
    x.of = of;
    x.part = part;
    uint32_t i, rest;
    const uint32_t group = p.b.div(of, i);
    x.qt = p.nqt - 1 - (int)group;
    x.bi = 0;
    if (p.b.d > 1) (void)p.b.div(i + ((p.clusters.div(group * p.b.d, rest) * 0x9E3779B1u) >> 16), x.bi);
    return x;
}
__device__ __forceinline__ Place place(const Params &p, uint32_t u) {
    uint32_t part = 0;
    return place_of(p, u < p.whole ? u : p.whole + p.parts.div(u - p.whole, part), part);
}

// What unit u needs from memory, for make_unit: asked for one unit ahead.
struct Ahead {
    Place at;
    int first, len;
};
__device__ __forceinline__ Ahead look(const Params &p, uint32_t u) {
    Ahead x;
    x.first = x.len = 0;
    if (u < p.units) {
        x.at = place(p, u);
        x.first = __ldg(p.a.first + x.at.bi);
        x.len = p.a.lens ? __ldg(p.a.lens + x.at.bi) : p.a.m;
    }
    return x;
}

// a: look(p, u)
__device__ __forceinline__ void make_unit(const Params &p, uint32_t u, const Ahead &a, Unit &x) {
    x.bi = (int)a.at.bi;
    x.part = (int)a.at.part;
    x.first = a.first;
    x.rows = max(0, min(a.len, p.a.m)) * p.a.h;
    x.r0 = a.at.qt * 2 * p.R;
    x.nw = x.nwp = x.nc = 0;
    x.wlo = 0;
    x.t0 = x.t1 = 0;
    x.clipped = false;
    if (x.r0 >= x.rows) return;
    uint32_t rest;
    const int64_t lo = (int64_t)x.first + p.h.div((uint32_t)x.r0, rest);
    const int64_t hi = (int64_t)x.first + p.h.div((uint32_t)min(x.r0 + 2 * p.R, x.rows) - 1, rest);
    if (hi < 0) return;
    if (p.a.window) x.wlo = (uint32_t)max((int64_t)0, lo - p.a.window + 1);
    int64_t end = hi + 1;
    if (!p.a.ring && end > p.cap) {
        end = p.cap;
        x.clipped = true;
    }
    x.nw = (int)max((int64_t)0, end - x.wlo);
    if (p.a.ratio) {
        int64_t nc = p.ratio.div((uint32_t)(hi + 1), rest);
        if (nc > p.cap - p.a.base) {
            x.clipped |= nc > 0;
            nc = max((int64_t)0, p.cap - p.a.base);
        }
        x.nc = (int)nc;
    }
    x.nwp = p.rows && x.nc ? (x.nw + BN - 1) / BN * BN : x.nw;      // WIDE: compressed rows begin a tile
    x.t1 = (int)((uint32_t)(x.nwp + x.nc + BN - 1) / BN);
    if (u >= p.whole) {                      // (at most 2^23 tiles, of at most 64 parts)
        x.t0 = (int)p.parts.div((uint32_t)(x.t1 * x.part), rest);
        x.t1 = (int)p.parts.div((uint32_t)(x.t1 * (x.part + 1)), rest);
    }
}

// What is left of a unit for whoever fetches its rows.
struct List {
    const int32_t *table;    // the sequence's pages
    uint32_t wlo;
    int nw, nwp, nv;         // window rows, where the compressed ones begin, where they end
};
__device__ __forceinline__ List list_of(const Params &p, const Unit &x) {
    return {p.a.block_table + (int64_t)x.bi * p.a.max_pages, x.wlo, x.nw, x.nwp, x.nwp + x.nc};
}

// Loads that leave v as it is unless `there`: nothing behind them selects, and so waits, before the value is needed.
__device__ __forceinline__ void ld_if(bool there, const int32_t *at, int &v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}" : "+r"(v) : "l"(at), "r"((int)there));
}
__device__ __forceinline__ void ld_if(bool there, const void *at, uint4 &v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
                 : "l"(at), "r"((int)there));
}

// Block table entry of the list's row v (-1 without one), and the row's place in its page (kNoRow behind the list's end).
constexpr uint32_t kNoRow = UINT32_MAX;
__device__ __forceinline__ int page_of(const Params &p, const List &x, int v, bool valid, uint32_t &off) {
    const bool row = valid && v < x.nv && (v < x.nw || v >= x.nwp);
    uint32_t r = v < x.nw ? x.wlo + (uint32_t)v : (uint32_t)(p.a.base + (v - x.nwp));
    if (v < x.nw && p.a.ring) p.ring.div(x.wlo + (uint32_t)v, r);
    const uint32_t pg = p.page.div(r, off);
    if (!row) off = kNoRow;
    int id = -1;
    ld_if(row && pg < (uint32_t)p.a.max_pages, x.table + pg, id);
    return id;
}
__device__ __forceinline__ bool is_page(const Params &p, int id) { return id >= 0 && id < p.a.pages; }

// Walks the tiles of this cluster's units.
struct TileIter {
    uint32_t u;
    int t, t1;
    List x;
    Ahead ahead;             // of unit u
    __device__ __forceinline__ bool valid() const { return t < t1; }
    __device__ __forceinline__ void seek(const Params &p, uint32_t step) {      // the first unit from u on with tiles
        while (u < p.units) {
            Unit unit;
            make_unit(p, u, ahead, unit);
            u += step;
            ahead = look(p, u);
            if (unit.t1 > unit.t0) {
                t = unit.t0;
                t1 = unit.t1;
                x = list_of(p, unit);
                return;
            }
        }
        t = t1 = 0;
    }
    __device__ __forceinline__ void start(const Params &p, uint32_t first, uint32_t step) {
        u = first;
        ahead = look(p, u);
        seek(p, step);
    }
    __device__ __forceinline__ void next(const Params &p, uint32_t step) {
        if (++t < t1) return;
        seek(p, step);
    }
};

// ---- single instructions ------------------------------------------------------------------------------------

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on this barrier in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}
// The same in the issuing CTA only.
__device__ __forceinline__ void commit_first(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// bf16 A and B, f32 accumulator; A K-major or MN-major, B K-major
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r != 0;
}
// Arrive on a barrier of any CTA of the cluster (an address from mapa).  For operands: they were written to this CTA's shared
// memory and fenced for the async proxy, and it is this SM's tensor core that reads them.  (At cluster scope a
// release waits for the codes under way too: 12000 cycles a tile instead of 3000.)
__device__ __forceinline__ void arrive_operand(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The same for what threads of the other CTA read, or write once it has been read: what this thread wrote or saw comes before what
// follows for who waits at cluster scope.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool test_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u16(uint32_t addr, uint16_t v) {
    asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
// TMA loads into this CTA's shared memory that count their bytes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int32_t x, int32_t y, int32_t z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ uint4 ld_codes(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bytes of v with their signs above them: 16-bit integers.
template <uint32_t kSel>
__device__ __forceinline__ uint32_t sign_extended(uint32_t v) {
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(v), "n"(kSel));
    return r;
}

// Sixteen codes times a power of two as bf16 pairs.  A code's exponent and mantissa bits, moved to a bf16's, are its value
// times 2^-120 (subnormals too), so one product with 2^(120 + k) makes it: b is that power's exponent field, 247 + k, or 0
// for zeros.  Two codes take a permutation and a mask in the integer pipe, and a shift and the product in the other (the bits put
// together from a word's nibbles took seven operations of the integer pipe for four codes).
__device__ __forceinline__ void widen16(const uint4 c, uint32_t b, uint32_t (&w)[8]) {
    const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
    const uint32_t scale = b * 0x00800080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // what the shift takes from the lower into the upper code is masked
        w[2 * i] = mul_bf16x2((sign_extended<0x9180>(cw[i]) * 16u) & 0x87f087f0u, scale);
        w[2 * i + 1] = mul_bf16x2((sign_extended<0xb3a2>(cw[i]) * 16u) & 0x87f087f0u, scale);
    }
}

// The exponents k of four blocks as widen16 takes them, 247 + min(k, 7); -128 stands for zeros.
constexpr uint32_t kZeros = 0x80808080u;
// A byte's top bit where k > 7.
__device__ __forceinline__ uint32_t above7(uint32_t four) { return ((four & 0x7f7f7f7fu) + 0x78787878u) & ~four & 0x80808080u; }
__device__ __forceinline__ uint32_t fields(uint32_t four, bool some_above7) {
    const uint32_t f = __vadd4(some_above7 ? __vmins4(four, 0x07070707u) : four, 0xf7f7f7f7u);
    // -128: the top bit and no other
    const uint32_t zero = four & ~((four & 0x7f7f7f7fu) + 0x7f7f7f7fu) & 0x80808080u;
    return zero ? f & ~((zero >> 7) * 255u) : f;
}

// Bits [lo, hi) of 64, both ends clamped to [0, 64].
__device__ __forceinline__ uint64_t bits(int lo, int hi) {
    const int a = max(0, min(64, lo)), z = max(0, min(64, hi));
    if (z <= a) return 0;
    return (z - a == 64 ? ~0ull : ((1ull << (z - a)) - 1)) << a;
}

// A head's sink in octaves, finite from above; a NaN stays one (in no reference, as fmaxf leaves it out, but in the denominator).
__device__ __forceinline__ float sink_log2(const Params &p, uint32_t hh) {
    const float v = __ldg(p.a.sink + hh) * kLog2e;
    return v > 1e37f ? 1e37f : v;
}

// What a role needs to wait, and to tell both CTAs to give up.
struct Ctl {
    uint32_t bars;
    volatile int *abort;
    uint32_t abort_own, abort_peer;
    __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
    __device__ __forceinline__ void give_up() const {
        st_cluster_u32(abort_own, 1);
        st_cluster_u32(abort_peer, 1);
    }
    // Every lane waits; false once a CTA of the cluster has given up.
    template <bool kCluster, uint64_t kLimit = kWaitLimitNs>
    __device__ __forceinline__ bool wait(int i, uint32_t phase) const {
        const uint32_t b = bar(i);
        bool ok = kCluster ? mbar_try_wait_cluster(b, phase & 1u) : mbar_try_wait(b, phase & 1u);
        if (!ok) {
            const uint64_t t0 = globaltimer_ns();
            for (uint32_t n = 1;; ++n) {
                ok = kCluster ? mbar_try_wait_cluster(b, phase & 1u) : mbar_try_wait(b, phase & 1u);
                if (ok) break;
                if ((n & 15u) == 0u) {
                    if (*abort) break;
                    if (globaltimer_ns() - t0 > kLimit) {
                        give_up();
                        break;
                    }
                }
            }
        }
        return __all_sync(kAll, ok);
    }
};

// ---- the kernel ---------------------------------------------------------------------------------------------

// kmap, vmap: WIDE: the workspace's rows, boxes of 64 rows by half of K's chunks and of 128 rows by two chunks
template <bool SPLIT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Roles<WIDE>::kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
    constexpr int W_WIDEN = Roles<WIDE>::kWiden, W_MMA = Roles<WIDE>::kMma, W_Q = Roles<WIDE>::kQ;
    constexpr int W_COPY = Roles<WIDE>::kCopy, W_LOAD = Roles<WIDE>::kLoad;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    uint8_t *ctl_mem = smem + SM_CTL;
    const uint32_t rank = cluster_ctarank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    Ctl c;
    c.bars = base + SM_CTL;
    c.abort = reinterpret_cast<volatile int *>(ctl_mem + C_ABORT);
    c.abort_own = mapa(c.bars + C_ABORT, rank);
    c.abort_peer = mapa(c.bars + C_ABORT, rank ^ 1u);
    auto first_bar = [&](int i) -> uint32_t { return mapa(c.bar(i), 0); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(c.bar(B_KFULL + i), WIDE ? 1 : 16);
            mbar_init(c.bar(B_KLOC + i), 8);
            mbar_init(c.bar(B_KFREE + i), WIDE ? 1 : 2);
            mbar_init(c.bar(B_VLOC + i), 1);
            mbar_init(c.bar(B_VFULL + i), WIDE ? 1 : 2);
            mbar_init(c.bar(B_VFREE + i), 1);
            mbar_init(c.bar(B_S + i), 1);
            mbar_init(c.bar(B_P + i), 8);
            mbar_init(c.bar(B_INV + i), 4);
            mbar_init(c.bar(B_INVFREE + i), 2 * Roles<WIDE>::kOut);
        }
        mbar_init(c.bar(B_Q), 1);
        mbar_init(c.bar(B_QFREE), 1);
        mbar_init(c.bar(B_O), 1);
        mbar_init(c.bar(B_OFREE), 2 * Roles<WIDE>::kOut);
        mbar_init(c.bar(B_RESCD), 2 * Roles<WIDE>::kOut);
        mbar_init(c.bar(B_SYNC), 1);
        mbar_init(c.bar(B_DRAIN), 1);
        *c.abort = (base & 1023u) != 0u;    // the operands' layout needs it aligned
        reinterpret_cast<int *>(ctl_mem + C_EVENT)[0] = 0;
        reinterpret_cast<int *>(ctl_mem + C_EVENT)[1] = 0;
        reinterpret_cast<int *>(ctl_mem + C_RESC)[0] = 0;
        reinterpret_cast<int *>(ctl_mem + C_RESC)[1] = 0;
        fence_mbar_init();
        grid_launch_dependents();
    }
    if (threadIdx.x < 256) reinterpret_cast<int16_t *>(ctl_mem + C_ALPHA)[threadIdx.x] = 0;
    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(c.bars + C_TMEM), "n"(TM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(ctl_mem + C_TMEM);
    // up to here this overlaps the kernel before it on the stream
    grid_dependency_wait();

    if (!WIDE && warp >= W_WIDEN && warp < W_MMA) {
        // ================================ widening: this CTA's 64 rows of the tile ================================
        // Warp w takes rows 8 w .. 8 w + 7, four lanes each.  Half h of K is chunks 2 h, 2 h + 1, 2 h + 4 and 2 h + 5 (half h of
        // V in either CTA); a step is one chunk, 16 codes a lane.  The next tile's codes are fetched into the registers of the
        // ones that have been widened.
        const int w = warp - W_WIDEN, q = lane & 3, r = 8 * w + (lane >> 2);
        const uint32_t full0 = first_bar(B_KFULL);
        // a lane's 16 values are 16-byte units 2 q and 2 q + 1 of the chunk: of two rows' lanes the swizzle makes one of each unit
        const uint32_t dst0 = base + SM_K + r * 128 + (((2 * q) ^ (r & 7)) << 4), flip = dst0 ^ 16u;
        const uint32_t sel = 0x4440u | (uint32_t)(q >> 1);               // this lane's exponent: of an even chunk; + 2: odd
        TileIter it;
        it.start(p, cid, ncl);
        uint4 code[2][4];
        bool bad = false;
        uint32_t off = 0;
        int id = -1;
        const uint8_t *row = p.a.codes + q * 16, *row_next = row;
        auto chunk_of = [](int h, int i) { return 2 * h + (i & 1) + 4 * (i >> 1); };
        auto fetch = [&](int h, int i) { code[h][i] = ld_codes(row + chunk_of(h, i) * 64); };
        auto look_up = [&]() { id = page_of(p, it.x, it.t * BN + HR * (int)rank + r, it.valid(), off); };
        // a row without a slot is read from slot 0 and widened to zeros
        auto exps_of = [&](const uint8_t *&at) -> uint4 {                 // of 128 values each
            const bool there = is_page(p, id);
            bad |= it.valid() && off != kNoRow && !there;
            const int64_t slot = there ? (int64_t)((uint32_t)id * p.page.d + off) : 0;
            at = p.a.codes + q * 16 + slot * D;
            uint4 e = make_uint4(kZeros, kZeros, kZeros, kZeros);
            ld_if(there, reinterpret_cast<const uint4 *>(p.a.exps) + slot, e);
            return e;
        };
        look_up();
        uint4 ex = exps_of(row);
#pragma unroll
        for (int i = 0; i < 8; ++i) fetch(i >> 2, i & 3);
        bool more = it.valid(), more_next = false;
        if (more) {
            it.next(p, ncl);
            more_next = it.valid();
            look_up();
        }
        uint4 ex_next = exps_of(row);                                     // from here on row is the next tile's
        for (uint32_t J = 0; more; ++J) {
            if (more_next) it.next(p, ncl);
            look_up();
            const bool slow = __any_sync(kAll, (above7(ex.x) | above7(ex.y) | above7(ex.z) | above7(ex.w)) != 0u);
            bool ok = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t e[2] = {h ? ex.y : ex.x, h ? ex.w : ex.z}, f[2] = {fields(e[0], slow), fields(e[1], slow)};
                ok = ok && c.wait<false>(B_KFREE + h, J + 1);
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t v[8];
                    widen16(code[h][i], __byte_perm(f[i >> 1], 0, sel + 2 * (i & 1)), v);
                    if (slow) {                  // the rest of powers above 2^127: 2^(k - 7)
                        const int k = (int)(__byte_perm(e[i >> 1], 0, sel + 2 * (i & 1)) << 24) >> 24;
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = mul_bf16x2(v[j], (uint32_t)(120 + max(k, 7)) * 0x00800080u);
                    }
                    st_shared_v4(dst0 + chunk_of(h, i) * K_CHUNK, v[0], v[1], v[2], v[3]);
                    st_shared_v4(flip + chunk_of(h, i) * K_CHUNK, v[4], v[5], v[6], v[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && !(p.stall && J == 0)) {
                    arrive_operand(full0 + 8 * h);
                    mbar_arrive(c.bar(B_KLOC + h));
                }
                // the page of the row after next is taken before loads are put behind it (they share a scoreboard), and the codes
                // are fetched behind the fence, which would wait for them
                if (h == 1) {
                    ex = ex_next;
                    ex_next = exps_of(row_next);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) fetch(h, i);
            }
            if (!ok) break;
            row = row_next;
            more = more_next;
            more_next = it.valid();
        }
        if (__any_sync(kAll, bad) && lane == 0) flag_status(p.a.status, DS_DEV_BAD_INDEX);
    } else if (warp >= W_MMA) {
        if constexpr (!WIDE) setmaxnreg_dec<REG_MMA>();
        if (warp == W_MMA) {
            // ======================================== MMA issue ========================================
            // The first CTA's warp walks the loop (its conditions are votes), an elected lane issues for both.  S of the next tile
            // goes before P V of this one when both can.
            if (rank == 0) {
                const uint32_t i_s = idesc(128, BN, false), i_pv = idesc(256, 2 * p.R, true);
                const uint64_t qd = smem_desc_sw128(base + SM_Q, 16, 1024), kd = smem_desc_sw128(base + SM_K, 16, 1024);
                const uint64_t vd = smem_desc_sw128(base + SM_V, V_CHUNK, 1024), pd = smem_desc_sw128(base + SM_P, 16, 1024);
                volatile int *cnt = reinterpret_cast<volatile int *>(ctl_mem + C_CNT);
                volatile int *resc = reinterpret_cast<volatile int *>(ctl_mem + C_RESC);
                auto done = [&](int b, uint32_t phase) -> bool { return __all_sync(kAll, mbar_test_wait(c.bar(b), phase & 1u)); };
                uint32_t u = cid;                      // S: its unit, that unit's tiles left, units begun
                int s_left = 0;
                uint32_t s_unit = 0, v_unit = 0;
                int v_left = 0;
                Ahead ahead = look(p, u);
                auto begin = [&]() {                   // the next unit with tiles
                    while (u < p.units) {
                        Unit x;
                        make_unit(p, u, ahead, x);
                        u += ncl;
                        ahead = look(p, u);
                        if (x.t1 > x.t0) {
                            s_left = x.t1 - x.t0;
                            __syncwarp();
                            cnt[s_unit & 3u] = s_left;
                            ++s_unit;
                            return;
                        }
                    }
                    s_left = 0;
                };
                uint32_t sJ = 0, vJ = 0, s_half = 0, v_half = 0, resc_n = 0, event = 0, idle = 0;   // event: phases of B_O
                bool s_first = true, v_first = true;
                uint64_t since = 0;
                begin();
                while (s_left > 0 || vJ < sJ) {
                    if (s_left > 0 && sJ - vJ < 2 && s_half == 0 && done(B_KFULL, sJ) && (!s_first || done(B_Q, s_unit - 1))) {
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const uint64_t at = (uint64_t)((((k >> 2) + (!WIDE && k >= 8 ? 2 : 0)) * K_CHUNK + (k & 3) * 32) >> 4);
                                mma_pair(tmem + TM_S + (sJ & 1u) * 64, qd + at, kd + at, i_s, k > 0);
                            }
                            commit_pair(c.bar(B_KFREE));
                        }
                        __syncwarp();
                        s_half = 1;
                        idle = 0;
                    } else if (s_half == 1 && done(B_KFULL + 1, sJ)) {
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const uint64_t at = (uint64_t)((((k >> 2) + (WIDE || k >= 8 ? 4 : 2)) * K_CHUNK + (k & 3) * 32) >> 4);
                                mma_pair(tmem + TM_S + (sJ & 1u) * 64, qd + at, kd + at, i_s, 1);
                            }
                            commit_pair(c.bar(B_S + (int)(sJ & 1u)));
                            commit_pair(c.bar(B_KFREE + 1));
                            if (s_left == 1) commit_pair(c.bar(B_QFREE));
                        }
                        __syncwarp();
                        s_half = 0;
                        s_first = false;
                        ++sJ;
                        if (--s_left == 0) {
                            begin();
                            s_first = true;
                        }
                        idle = 0;
                    } else if (vJ < sJ && v_half == 0 && done(B_P + (int)(vJ & 1u), vJ >> 1) && done(B_VFULL, vJ) &&
                               (!v_first || v_unit == 0 || done(B_OFREE, v_unit - 1))) {
                        if (v_first) v_left = cnt[v_unit & 3u];
                        tc_fence_after();
                        (void)test_wait_cluster(c.bar(B_P + (int)(vJ & 1u)), (vJ >> 1) & 1u);   // again, for what the other CTA wrote here
                        if (__any_sync(kAll, resc[vJ & 1u] == (int)(vJ + 1))) {
                            // a reference has moved: O^T of the tiles before this one is scaled first
                            if (elect_one()) commit_first(c.bar(B_SYNC));
                            __syncwarp();
                            if (!c.wait<true>(B_SYNC, resc_n)) break;
                            if (lane < 2) {
                                st_cluster_u32(mapa(c.bars + C_EVENT + 4 * (event & 1u), (uint32_t)lane), 2 * (event + 1) + (vJ & 1u));
                                arrive_cluster(mapa(c.bar(B_O), (uint32_t)lane));
                            }
                            ++event;
                            if (!c.wait<true>(B_RESCD, resc_n)) break;
                            ++resc_n;
                            tc_fence_after();
                        }
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_pair(tmem + TM_O, vd + (uint64_t)((k * 2048) >> 4),
                                         pd + (uint64_t)(((vJ & 1u) * P_BYTES + (k >> 2) * K_CHUNK + (k & 3) * 32) >> 4), i_pv,
                                         k > 0 || !v_first);
                            commit_pair(c.bar(B_VFREE));
                        }
                        __syncwarp();
                        v_half = 1;
                        idle = 0;
                    } else if (v_half == 1 && done(B_VFULL + 1, vJ)) {
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                mma_pair(tmem + TM_O + 128, vd + (uint64_t)((2 * V_CHUNK + k * 2048) >> 4),
                                         pd + (uint64_t)(((vJ & 1u) * P_BYTES + (k >> 2) * K_CHUNK + (k & 3) * 32) >> 4), i_pv,
                                         k > 0 || !v_first);
                            commit_pair(c.bar(B_VFREE + 1));
                            if (v_left == 1) commit_pair(c.bar(B_O));
                        }
                        __syncwarp();
                        v_half = 0;
                        v_first = false;
                        ++vJ;
                        if (--v_left == 0) {
                            ++v_unit;
                            ++event;
                            v_first = true;
                        }
                        idle = 0;
                    } else {
                        __nanosleep(20);
                        if ((++idle & 63u) == 0u) {
                            const uint64_t now = globaltimer_ns();
                            if (idle == 64u) since = now;
                            else if (now - since > kWaitLimitNs) c.give_up();
                            if (__any_sync(kAll, *c.abort != 0)) break;
                        }
                    }
                }
                if (elect_one()) commit_pair(c.bar(B_DRAIN));
                __syncwarp();
            }
        } else if (warp == W_Q) {
            // ======================================== q by TMA ========================================
            if (lane == 0) {
                const uint32_t full = first_bar(B_Q);
                uint32_t n = 0;
                Ahead ahead = look(p, cid);
                for (uint32_t u = cid; u < p.units; u += ncl) {
                    Unit x;
                    make_unit(p, u, ahead, x);
                    ahead = look(p, u + ncl);
                    if (x.t1 <= x.t0) continue;
                    if (!mbar_wait(c.bar(B_QFREE), (n & 1u) ^ 1u, c.abort, kUnitLimitNs)) {
                        c.give_up();
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(c.bar(B_Q), (uint32_t)(2 * p.R * D * 2));    // both CTAs'
                    const int32_t y = (int32_t)((int64_t)x.bi * p.a.m * p.a.h + x.r0 + (int)rank * p.R);
                    for (int ch = 0; ch < 8; ++ch) tma_load_2d(base + SM_Q + ch * K_CHUNK, &qmap, ch * 64, y, full);
                    ++n;
                }
            }
            __syncwarp();
        } else if (WIDE) {
            // ======================= K (warp W_LOAD) and V (the next one) by TMA, in halves =======================
            const bool isv = warp != W_LOAD;
            if (lane == 0) {
                const CUtensorMap *map = isv ? &vmap : &kmap;
                const uint32_t full = first_bar(isv ? B_VFULL : B_KFULL);
                const int free0 = isv ? B_VFREE : B_KFREE;
                const uint32_t dst = base + (isv ? SM_V : SM_K);
                uint32_t J = 0;
                Ahead ahead = look(p, cid);
                for (uint32_t u = cid; u < p.units; u += ncl) {
                    Unit x;
                    make_unit(p, u, ahead, x);
                    ahead = look(p, u + ncl);
                    const int64_t wbase = p.a.window ? max((int64_t)0, (int64_t)x.first - p.a.window + 1) : 0;
                    bool ok = true;
                    for (int t = x.t0; t < x.t1; ++t, ++J) {
                        const int v0 = t * BN, w0 = (int)(x.wlo - wbase) + v0;
                        const int y = x.bi * (p.wrows + p.crows) + (v0 < x.nwp ? w0 : p.wrows + v0 - x.nwp) + (isv ? 0 : HR * (int)rank);
                        for (int h = 0; h < 2; ++h) {
                            ok = ok && mbar_wait(c.bar(free0 + h), (J & 1u) ^ 1u, c.abort, kWaitLimitNs);
                            if (!ok) break;
                            if (rank == 0 && !(p.stall && J == 0)) mbar_arrive_expect_tx(c.bar((isv ? B_VFULL : B_KFULL) + h), 8 * K_CHUNK);
                            tma_load_3d(dst + h * 4 * K_CHUNK, map, 0, y, isv ? 4 * (int)rank + 2 * h : 4 * h, full + 8 * h);
                        }
                        if (!ok) break;
                    }
                    if (!ok) {
                        c.give_up();
                        break;
                    }
                }
            }
            __syncwarp();
        } else {
            // ================================ half h of K to both CTAs' V ================================
            // The copy engine takes the other CTA's chunks, this warp its own (the engine with both: 2 us a tile, 1 us each 32 KB).
            const int h = warp - W_COPY;
            const uint32_t vfull = first_bar(B_VFULL + h), to = rank ^ 1u;
            const uint32_t from = base + SM_K + (4 * rank + 2 * h) * K_CHUNK + lane * 16;
            const uint32_t own = base + SM_V + 2 * h * V_CHUNK + rank * K_CHUNK + lane * 16;
            TileIter it;
            it.start(p, cid, ncl);
            for (uint32_t J = 0; it.valid(); ++J, it.next(p, ncl)) {
                if (!c.wait<false>(B_KLOC + h, J) || !c.wait<false>(B_VFREE + h, J + 1)) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(c.bar(B_VLOC + h), 2 * K_CHUNK);   // the other CTA's rows
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        bulk_copy_to_peer(mapa(base + SM_V + (2 * h + i) * V_CHUNK + rank * K_CHUNK, to),
                                          base + SM_K + (4 * to + 2 * h + i) * K_CHUNK, K_CHUNK, mapa(c.bar(B_VLOC + h), to));
                    bulk_commit_group();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll 1
                    for (int k = 0; k < K_CHUNK; k += 2048) {
                        float4 x[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[j] = ld_shared_v4(from + i * K_CHUNK + k + j * 512);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            st_shared_v4(own + i * V_CHUNK + k + j * 512, __float_as_uint(x[j].x), __float_as_uint(x[j].y), __float_as_uint(x[j].z),
                                         __float_as_uint(x[j].w));
                    }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bulk_wait_read_all();
                    mbar_arrive(c.bar(B_KFREE + h));
                }
                if (!c.wait<false>(B_VLOC + h, J)) break;
                if (lane == 0) arrive_operand(vfull);
            }
            if (lane == 0) bulk_wait_all();                                  // nothing may land after the CTAs are gone
            __syncwarp();
        }
    } else if (warp < W_OUT) {
        if constexpr (!WIDE) setmaxnreg_inc<REG_SOFTMAX>();
        // ======================================== softmax ========================================
        // Lane r of the scores (warps 0 and 1: r < 64) has query r and the tile's rows 0-63, lane r + 64 the same query and rows
        // 64-127; the two threads share the reference through shared memory and a barrier of their two warps.
        const int half = warp >> 1, row = (warp & 1) * 32 + lane;
        const uint32_t tm = tmem + ((uint32_t)(warp * 32) << 16) + TM_S;
        const uint32_t pfull[2] = {first_bar(B_P), first_bar(B_P + 1)};
        const uint32_t resc = mapa(c.bars + C_RESC, 0);
        float *xch = reinterpret_cast<float *>(ctl_mem + C_XCH);
        const float scale = p.scale_log2 == 0.0f ? 1.0f : fabsf(p.scale_log2);   // its sign, or a 0, goes to the scores
        const bool idle_warp = (warp & 1) * 32 >= p.R;          // no query of these 32
        bool dead = false, bad = false;
        uint32_t J = 0, unit = 0, ex = 0;                       // tiles, whole units with tiles, exchanges
        uint32_t lowered = 0;                                   // bit J & 1: this thread's entry of alpha is not 0
        auto exchange = [&](float v) -> float {                 // the other thread's value
            float *x = xch + (ex & 1u) * 128;
            ++ex;
            x[half * 64 + row] = v;
            named_bar_sync(1 + (warp & 1), 64);
            return x[(half ^ 1) * 64 + row];
        };
        Ahead ahead = look(p, cid);
        for (uint32_t u = cid; u < p.units; u += ncl) {
            Unit x;
            make_unit(p, u, ahead, x);
            ahead = look(p, u + ncl);
            const int rq = (int)rank * p.R + row;               // query row of the unit
            const bool live = row < p.R && x.r0 + rq < x.rows;
            uint32_t hh = 0;
            const int64_t pos = (int64_t)x.first + (live ? p.h.div((uint32_t)(x.r0 + rq), hh) : 0);
            bad |= (live && pos < 0) || x.clipped;
            const float sink2 = live ? sink_log2(p, hh) : 0.0f;
            // rows [a0, a1) and [nwp, c1) of the list
            int a0 = 0, a1 = 0, c1 = 0;
            if (live && pos >= 0) {
                a0 = p.a.window ? (int)max((int64_t)0, pos - p.a.window + 1 - x.wlo) : 0;
                a1 = (int)min(pos + 1 - x.wlo, (int64_t)x.nw);
                uint32_t rest;
                c1 = x.nwp + (p.a.ratio ? (int)min(p.ratio.div((uint32_t)(pos + 1), rest), (uint32_t)x.nc) : 0);
            }
            const List list = list_of(p, x);
            float ref = sink2 - 64.0f, l = 0.0f;
            bool set = false;
            for (int t = x.t0; t < x.t1; ++t, ++J) {
                const int v0 = t * BN + half * 64;
                uint64_t mask = 0;
                bool told = false;                              // this warp has stored what threads of the other CTA read
                if (!idle_warp) {
                    uint32_t off;
                    const bool there0 = is_page(p, page_of(p, list, v0 + lane, true, off));
                    const bool there1 = is_page(p, page_of(p, list, v0 + 32 + lane, true, off));
                    const uint64_t there = (uint64_t)__ballot_sync(kAll, there0) | ((uint64_t)__ballot_sync(kAll, there1) << 32);
                    mask = there & (bits(a0 - v0, a1 - v0) | bits(x.nwp - v0, c1 - v0));
                }
                if (!dead) dead = !c.wait<false>(B_S + (int)(J & 1u), J >> 1);
                if (!idle_warp) {
                    tc_fence_after();
                    uint32_t s[2][32];
                    tmem_ld32(tm + (J & 1u) * 64, s[0]);
                    tmem_ld32(tm + (J & 1u) * 64 + 32, s[1]);
                    tmem_ld_wait(s);
                    tc_fence_before();
                    const bool whole = __all_sync(kAll, mask == ~0ull);
                    if (p.scale_log2 <= 0.0f) {
                        const float f = p.scale_log2 < 0.0f ? -1.0f : 0.0f;
#pragma unroll
                        for (int g = 0; g < 64; ++g) s[g >> 5][g & 31] = __float_as_uint(__uint_as_float(s[g >> 5][g & 31]) * f);
                    }
                    if (!whole) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const uint32_t mk = (uint32_t)(mask >> (32 * g));
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((mk >> i) & 1u)) s[g][i] = 0xff800000u;
                        }
                    }
                    float mm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};     // four chains: a chain of 32 is 0.1 us
#pragma unroll
                    for (int i = 0; i < 64; i += 2)
                        mm[(i >> 1) & 3] = max3(mm[(i >> 1) & 3], __uint_as_float(s[i >> 5][i & 31]), __uint_as_float(s[i >> 5][(i & 31) + 1]));
                    float m = fmaxf(max3(mm[0], mm[1], mm[2]), mm[3]);
                    m = m == -INFINITY ? m : m * scale;
                    m = fmaxf(m, exchange(m));
                    const int q = (int)rank * p.R + row;
                    const uint32_t alpha = c.bars + C_ALPHA + ((J & 1u) * 128 + q) * 2;
                    float up = 0.0f;
                    if (!set) {
                        if (m > -INFINITY) {
                            ref = fmaxf(ref, m + kSlack);
                            set = true;
                        }
                    } else if (m > ref) {
                        up = fminf(ceilf(m - ref) + kSlack, 16384.0f);
                        ref = up < 16384.0f ? ref + up : m + kSlack;
                        l *= ex2(-up);
                    }
                    // alpha's entries of this tile were last used two tiles ago: one that was not 0 then is set back
                    const bool tell = half == 0 && row < p.R && (up > 0.0f || ((lowered >> (J & 1u)) & 1u));
                    told = __any_sync(kAll, tell);
                    if (tell) {
                        st_cluster_u16(mapa(alpha, 0), (uint16_t)up);
                        st_cluster_u16(mapa(alpha, 1), (uint16_t)up);
                        lowered = (lowered & ~(1u << (J & 1u))) | ((up > 0.0f ? 1u : 0u) << (J & 1u));
                        if (up > 0.0f) st_cluster_u32(resc + (J & 1u) * 4, J + 1);
                    }
                    const uint64_t neg = pair(set ? -ref : 0.0f, set ? -ref : 0.0f), scale2 = pair(scale, scale);
                    uint64_t sum = pair(0.0f, 0.0f);
                    const uint32_t at = base + SM_P + (J & 1u) * P_BYTES + half * K_CHUNK + row * 128;
#pragma unroll
                    for (int g = 0; g < 2; ++g)
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float e0, e1;
                                unpair(fma2(pair(__uint_as_float(s[g][i + 2 * j]), __uint_as_float(s[g][i + 2 * j + 1])), scale2, neg), e0, e1);
                                e0 = ex2(e0);
                                e1 = ex2(e1);
                                sum = add2(sum, pair(e0, e1));
                                w[j] = pack_bf16x2(e0, e1);
                            }
                            st_shared_v4(at + (((uint32_t)(g * 4 + i / 8) ^ (row & 7)) << 4), w[0], w[1], w[2], w[3]);
                        }
                    float la, lb;
                    unpair(sum, la, lb);
                    l += la + lb;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if (told) arrive_cluster(pfull[J & 1u]);
                    else arrive_operand(pfull[J & 1u]);
                }
            }
            const bool split = SPLIT && u >= p.whole;           // a part: its reference and sum go to the workspace
            float *st = split ? p.ws + ((size_t)(u - p.whole) * (D + 2) + D) * (2 * p.R) + 2 * rq : nullptr;
            if (x.t1 == x.t0) {
                if (split && live && half == 0) {
                    st[0] = -INFINITY;
                    st[1] = 0.0f;
                }
                continue;
            }
            if (!idle_warp) l += exchange(l);
            if (split) {
                if (live && half == 0) {
                    st[0] = ref;
                    st[1] = l;
                }
                continue;
            }
            if (half == 0) {
                // the factors of two units ago have been read: units of one tile end faster than outputs are written
                if (!dead) dead = !c.wait<true>(B_INVFREE + (int)(unit & 1u), (unit >> 1) + 1);
                if (row < p.R) {
                    const float inv = l > 0.0f ? 1.0f / (l + ex2(sink2 - ref)) : (l == 0.0f ? 0.0f : l);
                    const uint32_t at = c.bars + C_INV + ((unit & 1u) * 128 + rq) * 4;
                    st_cluster_u32(mapa(at, 0), __float_as_uint(inv));
                    st_cluster_u32(mapa(at, 1), __float_as_uint(inv));
                }
                __syncwarp();
                if (lane < 2) arrive_cluster(mapa(c.bar(B_INV + (int)(unit & 1u)), (uint32_t)lane));
            }
            ++unit;
        }
        if (__any_sync(kAll, bad) && lane == 0) flag_status(p.a.status, DS_DEV_BAD_INDEX);
    } else {
        if constexpr (!WIDE) setmaxnreg_inc<REG_OUT>();
        // ================================== output, and O^T's rescaling ==================================
        // Thread (warp w, lane) has d = 256 rank + 128 v + 32 w + lane of every query: column q of O^T's block v.
        // Of eight warps, those of one lane quarter share it by queries, 64 each: the rotation falls on two quarters of the second
        // block, and a warp that had all of that kept O^T 1.7 us longer (prompt of 4096 tokens: 384 us, 339 without a rotation).
        const int w = warp & 3, q0 = WIDE ? ((warp - W_OUT) >> 2) * 64 : 0, q1 = WIDE ? q0 + 64 : 128;   // its queries
        const uint32_t tm = tmem + ((uint32_t)(w * 32) << 16) + TM_O;
        const uint32_t free_bar = first_bar(B_OFREE), resc_bar = first_bar(B_RESCD);
        const int16_t *alpha = reinterpret_cast<const int16_t *>(ctl_mem + C_ALPHA);
        const int nq = 2 * p.R;
        const int d0 = 256 * (int)rank + 32 * w + lane;
        uint32_t unit = 0, event = 0;
        bool bad = false, ok = true;
        Ahead ahead = look(p, cid);
        for (uint32_t u = cid; u < p.units && ok; u += ncl) {
            Unit x;
            make_unit(p, u, ahead, x);
            ahead = look(p, u + ncl);
            const bool some = x.t1 > x.t0, split = SPLIT && u >= p.whole;
            if (split && !some) continue;
            if (some) {
                for (;; ++event) {
                    ok = c.wait<true, kUnitLimitNs>(B_O, event);
                    if (!ok) break;
                    const uint32_t e = *reinterpret_cast<volatile uint32_t *>(ctl_mem + C_EVENT + 4 * (event & 1u));
                    if (e >> 1 != event + 1) break;
                    tc_fence_after();
                    for (int g = q0; g < min(nq, q1); g += 32) {
                        const int up = *reinterpret_cast<const volatile int16_t *>(alpha + (e & 1u) * 128 + g + lane);
                        if (!__any_sync(kAll, up != 0)) continue;
                        const float f = ex2(-(float)up);
#pragma unroll 1
                        for (int v = 0; v < 2; ++v) {
                            uint32_t r[32];
                            tmem_ld32(tm + v * 128 + g, r);
                            tmem_ld_wait(r);
#pragma unroll
                            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * __shfl_sync(kAll, f, j));
                            tmem_st32(tm + v * 128 + g, r);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(resc_bar);
                }
                ++event;
                if (ok && !split) ok = c.wait<true>(B_INV + (int)(unit & 1u), unit >> 1);
                if (!ok) break;
                tc_fence_after();
            }
            const int there = x.rows - x.r0;                 // queries of this unit
            const float *inv = reinterpret_cast<const float *>(ctl_mem + C_INV) + (unit & 1u) * 128;
            uint16_t *o = p.a.o + ((int64_t)x.bi * p.a.m * p.a.h + x.r0) * D;
            uint32_t hh;
            float *part = split ? p.ws + (size_t)(u - p.whole) * (D + 2) * nq : nullptr;
            if (!some) {                                     // nothing seen: zeros, which no rotation changes
                if (there <= 0) continue;
                for (int q = q0; q < min(min(nq, q1), there); ++q)
                    for (int v = 0; v < 2; ++v) o[(int64_t)q * D + d0 + 128 * v] = 0;
                const int64_t pos0 = (int64_t)x.first + p.h.div((uint32_t)x.r0, hh);
                const int64_t pos1 = (int64_t)x.first + p.h.div((uint32_t)(x.r0 + min(nq, there) - 1), hh);
                bad |= p.a.rd > 0 && (pos0 < 0 || pos1 >= p.a.table_rows);
                continue;
            }
            // a token's angles: table rows from its position on; tokens [in0, in1) of the unit's lie in the table
            const int64_t pos0 = (int64_t)x.first + p.h.div((uint32_t)x.r0, hh);
            const int in0 = pos0 < 0 ? (int)min(-pos0, (int64_t)128) : 0;
            const int in1 = (int)max((int64_t)0, min(p.a.table_rows - pos0, (int64_t)129));
            const int half_rd = p.a.rd / 2;
            // 32 queries of a block at a time: issuing a load of tensor memory takes a warp some 150 cycles whatever its size
            // (steps of eight queries took 540 cycles each, a unit 4.4 us).
            constexpr int G = 32;
            const int last = ((min(min(nq, q1), there) + G - 1) / G - 1) * G;
            if (last < q0) {                                 // none of its queries is there
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_operand(free_bar);
            }
#pragma unroll 1
            for (int v = 0; v < 2; ++v) {
                const int d = d0 + 128 * v, pair = (d - (D - p.a.rd)) >> 1;
                const bool rot = !split && p.a.rd > 0 && 256 * (int)rank + 128 * v + 32 * w + 31 >= D - p.a.rd;
                const bool odd = d & 1;
                const float2 *angles = rot && pair >= 0 ? p.a.table + pos0 * half_rd + pair : nullptr;
                uint32_t head;                               // the next query's head and token
                int tok = (int)p.h.div(hh + (uint32_t)q0, head), at = (int)head;
                auto angle = [&]() -> float2 {
                    const bool in = tok >= in0 && tok < in1;
                    bad |= !in;
                    float2 cs = in && angles ? __ldg(angles) : make_float2(1.0f, 0.0f);
                    if (odd) cs.y = -cs.y;
                    return cs;
                };
                auto advance = [&](int n) {
                    if ((at += n) == (int)p.h.d) {
                        at = 0;
                        ++tok;
                        if (angles) angles += half_rd;
                    }
                };
                if (angles) angles += tok * half_rd;
                uint16_t *to = o + d + q0 * D;
                float *top = split ? part + d + q0 * D : nullptr;
#pragma unroll 1
                for (int g = q0; g <= last; g += G) {
                    uint32_t r[G];
                    tmem_ld32(tm + v * 128 + g, r);
                    float2 c8[4];                            // angles of eight queries that one token has
                    uint32_t ones = 0;
                    if (rot && at + G <= (int)p.h.d) {
                        c8[0] = c8[1] = c8[2] = c8[3] = angle();
                        advance(G);
                        ones = 15;
                    }
                    tmem_ld_wait(r);
                    if (g == last && v == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_operand(free_bar);
                    }
                    if (split) {
#pragma unroll
                        for (int j = 0; j < G; ++j)
                            if (g + j < there) top[j * D] = __uint_as_float(r[j]);
                        top += G * D;
                        continue;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int left = there - g - 8 * e;
                        const float4 fa = *reinterpret_cast<const float4 *>(inv + g + 8 * e);
                        const float4 fb = *reinterpret_cast<const float4 *>(inv + g + 8 * e + 4);
                        const float f[8] = {fa.x, fa.y, fa.z, fa.w, fb.x, fb.y, fb.z, fb.w};
                        float x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[8 * e + j]) * f[j];
                        if (rot && left > 0) {               // pairs are neighbouring lanes
                            if (!((ones >> e) & 1u) && at + 8 <= (int)p.h.d) {
                                c8[e] = angle();
                                advance(8);
                                ones |= 1u << e;
                            }
                            if ((ones >> e) & 1u) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) x[j] = x[j] * c8[e].x + __shfl_xor_sync(kAll, x[j], 1) * c8[e].y;
                            } else {                         // several tokens in eight queries
                                float2 cs[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    cs[j] = j < left ? angle() : make_float2(1.0f, 0.0f);
                                    advance(1);
                                }
#pragma unroll
                                for (int j = 0; j < 8; ++j) x[j] = x[j] * cs[j].x + __shfl_xor_sync(kAll, x[j], 1) * cs[j].y;
                            }
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < left) to[(8 * e + j) * D] = __bfloat16_as_ushort(__float2bfloat16_rn(x[j]));
                    }
                    to += G * D;
                }
            }
            if (!split) {                                    // (units without rows have gone on above)
                __syncwarp();
                // both CTAs' softmax threads write the next ones.  (At cluster scope this waits for the output's stores, 0.3 us where nothing
                // is left to do: not behind the last unit, for which nobody waits.)
                if (lane < 2 && u + ncl < p.units) arrive_cluster(mapa(c.bar(B_INVFREE + (int)(unit & 1u)), (uint32_t)lane));
                ++unit;
            }
        }
        if (__any_sync(kAll, bad) && lane == 0) flag_status(p.a.status, DS_DEV_BAD_INDEX);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (*c.abort) {
        if (threadIdx.x == 0) flag_status(p.a.status, DS_DEV_TIMEOUT);
        // loads that were issued before somebody gave up land within microseconds
        for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 2000000ull;) {
        }
    }
    // no MMA and no commit is under way in either CTA once this has passed
    if (warp == W_MMA) {
        mbar_wait_drain(c.bar(B_DRAIN), 0, 2 * kWaitLimitNs);
        __syncwarp();
    }
    __syncthreads();
    cluster_sync();
    if (warp == W_MMA)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(TM_COLS) : "memory");
}

// ---- WIDE: the rows that the queries see, in bf16 ----------------------------------------------------------------

constexpr int kRowsBlock = 64;

// Block (x, bi): 64 rows of sequence bi, of positions from the first that a query sees on, then compressed ones.  Behind each
// kind's last row come 128 of zeros: a tile's end is read, and P V adds 0 times what it holds.
__global__ void __launch_bounds__(256) chunk_rows_kernel(const __grid_constant__ Params p) {
    if (threadIdx.x == 0) grid_launch_dependents();
    grid_dependency_wait();
    __shared__ int slot[kRowsBlock];         // -1: zeros, -2: nothing
    const int bi = blockIdx.y, wblocks = (p.wrows + kRowsBlock - 1) / kRowsBlock;
    const bool comp = (int)blockIdx.x >= wblocks;
    const int i0 = ((int)blockIdx.x - (comp ? wblocks : 0)) * kRowsBlock;
    if ((int)threadIdx.x < kRowsBlock) {
        const int n = p.a.lens ? max(0, min(__ldg(p.a.lens + bi), p.a.m)) : p.a.m, i = i0 + threadIdx.x;
        const int64_t first = __ldg(p.a.first + bi), end = first + n;          // positions below end are seen
        const int64_t wbase = p.a.window ? max((int64_t)0, first - p.a.window + 1) : 0;
        uint32_t rest;
        int64_t count = comp ? (end > 0 ? (int64_t)p.ratio.div((uint32_t)end, rest) : 0) : max((int64_t)0, end - wbase);
        if (comp) count = min(count, max((int64_t)0, p.cap - p.a.base));
        else if (!p.a.ring) count = min(count, max((int64_t)0, p.cap - wbase));
        int at = -2;
        if (n > 0 && i < (comp ? p.crows : p.wrows) && i < count + BN) {
            at = -1;
            if (i < count) {
                uint32_t r = comp ? (uint32_t)(p.a.base + i) : (uint32_t)(wbase + i), off;
                if (!comp && p.a.ring) p.ring.div((uint32_t)(wbase + i), r);
                const uint32_t pg = p.page.div(r, off);
                const int id = pg < (uint32_t)p.a.max_pages ? __ldg(p.a.block_table + (int64_t)bi * p.a.max_pages + pg) : -1;
                if (is_page(p, id)) at = (int)((uint32_t)id * p.page.d + off);
                else flag_status(p.a.status, DS_DEV_BAD_INDEX);
            }
        }
        slot[threadIdx.x] = at;
    }
    __syncthreads();
    uint4 *out = reinterpret_cast<uint4 *>(p.rows) + ((int64_t)bi * (p.wrows + p.crows) + (comp ? p.wrows : 0) + i0) * (D / 8);
    constexpr int kSteps = 4;
#pragma unroll 1
    for (int u0 = threadIdx.x; u0 < kRowsBlock * (D / 8); u0 += 256 * kSteps) {
        uint2 code[kSteps];
        int k[kSteps], at[kSteps];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const int u = u0 + 256 * j, ch = u % (D / 8);
            at[j] = slot[u / (D / 8)];
            code[j] = make_uint2(0, 0);
            k[j] = -128;
            if (at[j] >= 0) {
                code[j] = __ldg(reinterpret_cast<const uint2 *>(p.a.codes) + (int64_t)at[j] * (D / 8) + ch);
                k[j] = __ldg(p.a.exps + (int64_t)at[j] * (D / 32) + (ch >> 2));
            }
        }
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            if (at[j] == -2) continue;
            uint32_t w[8];
            widen16(make_uint4(code[j].x, code[j].y, 0, 0), k[j] == -128 ? 0u : (uint32_t)(247 + min(k[j], 7)), w);
            if (k[j] > 7) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = mul_bf16x2(w[i], (uint32_t)(120 + k[j]) * 0x00800080u);
            }
            out[u0 + 256 * j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---- parts of a unit joined ------------------------------------------------------------------------------------

constexpr int kMaxParts = 64;
// Query tiles of a sequence from which its rows are widened once, in a pass of their own: with three tiles that takes 0.87 of
// the time (32 sequences, 3 tokens of 128 heads, 2176 rows: 74 us instead of 85), with two 1.02 (64 sequences, 2 tokens: 117
// instead of 114), with one 1.3 (32 sequences of 4224 rows: 78 instead of 59 us; 128 rows: 19.0 instead of 13.6).
constexpr int kWideTiles = 3;

// One query row a block; thread i has values 4 i .. 4 i + 3.  Each part has its reference, its sum and its O^T, and kFlight parts
// are read at once.  With few parts 16 in flight cost occupancy (two parts of 32 sequences: 62 us a call instead of 58, nine of 16
// sequences 105 instead of 103), with many they save latency (44 parts: 21 instead of 25, 18 of four sequences 18 instead of 22).
constexpr int kManyParts = 12;
template <int kFlight>
__global__ void __launch_bounds__(128) chunk_merge_kernel(const __grid_constant__ Params p) {
    grid_dependency_wait();
    const uint32_t tile = blockIdx.x;               // of those that are in parts
    const int q = blockIdx.y, lane = threadIdx.x & 31;
    const Place pl = place_of(p, p.whole + tile, 0);
    const uint32_t bi = pl.bi;
    const int qt = pl.qt;
    uint32_t hh;
    const int n = p.a.lens ? max(0, min(__ldg(p.a.lens + bi), p.a.m)) : p.a.m, r = qt * 2 * p.R + q;
    if (r >= n * p.a.h) return;
    const int64_t pos = (int64_t)__ldg(p.a.first + bi) + p.h.div((uint32_t)r, hh);
    const int np = (int)p.parts.d;
    const size_t slot = (size_t)(D + 2) * (2 * p.R);
    const float *ws = p.ws + (size_t)tile * np * slot;
    float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = lane + 32 * i;
        if (k < np) {
            const float2 st = *reinterpret_cast<const float2 *>(ws + k * slot + (size_t)D * (2 * p.R) + 2 * q);
            l[i] = st.y;
            ref[i] = st.y == 0.0f ? -INFINITY : st.x;
        }
    }
    float top = fmaxf(ref[0], ref[1]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    float wgt[2], den = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        wgt[i] = l[i] == 0.0f ? 0.0f : ex2(ref[i] - top);
        den += wgt[i] * l[i];
    }
    den = rows::row_sum<32>(den);
    const float sink2 = sink_log2(p, hh);
    const float inv = den == 0.0f ? 0.0f : 1.0f / (den + ex2(sink2 - top));
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float *src = ws + (size_t)q * D + 4 * threadIdx.x;
    for (int k0 = 0; k0 < np; k0 += kFlight) {
        float f[kFlight];
        float4 v[kFlight];
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            const int k = k0 + i;
            f[i] = __shfl_sync(kAll, k < 32 ? wgt[0] : wgt[1], k & 31);
            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k < np && f[i] != 0.0f) v[i] = __ldcg(reinterpret_cast<const float4 *>(src + k * slot));
            else f[i] = 0.0f;                       // (a part without rows wrote none)
        }
#pragma unroll
        for (int i = 0; i < kFlight; ++i) {
            acc.x = fmaf(f[i], v[i].x, acc.x);
            acc.y = fmaf(f[i], v[i].y, acc.y);
            acc.z = fmaf(f[i], v[i].z, acc.z);
            acc.w = fmaf(f[i], v[i].w, acc.w);
        }
    }
    acc.x *= inv;
    acc.y *= inv;
    acc.z *= inv;
    acc.w *= inv;
    const int j = 4 * (int)threadIdx.x - (D - p.a.rd);
    if (p.a.rd) {
        if (pos >= 0 && pos < p.a.table_rows) {
            if (j >= 0) {
                const float2 *cs = p.a.table + pos * (p.a.rd / 2) + j / 2;
                const float2 c0 = __ldg(cs), c1 = __ldg(cs + 1);
                acc = make_float4(acc.x * c0.x + acc.y * c0.y, acc.y * c0.x - acc.x * c0.y, acc.z * c1.x + acc.w * c1.y,
                                  acc.w * c1.x - acc.z * c1.y);
            }
        } else if (threadIdx.x == 0) {
            flag_status(p.a.status, DS_DEV_BAD_INDEX);
        }
    }
    reinterpret_cast<uint2 *>(p.a.o + (((int64_t)bi * p.a.m * p.a.h + r) * D))[threadIdx.x] =
        make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

// ---- host side --------------------------------------------------------------------------------------------------

constexpr int kMaxDev = 64;
int g_clusters[kMaxDev];
std::mutex g_mutex;
std::atomic<int> g_test_stall{0};

// Clusters that run at once on the current device, 0 when the kernel cannot be configured.
int max_clusters(int dev) {
    if (dev < 0 || dev >= kMaxDev) return 0;
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_clusters[dev]) return g_clusters[dev];
    int least = INT32_MAX, sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    auto add = [&](const void *k, int threads) {
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess) return false;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(sms / 2 * 2), 1, 1);
        cfg.blockDim = dim3((unsigned)threads, 1, 1);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return false;
        least = std::min(least, n);
        return true;
    };
    if (!add((const void *)chunk_attn_kernel<false, false>, Roles<false>::kThreads) ||
        !add((const void *)chunk_attn_kernel<true, false>, Roles<false>::kThreads) ||
        !add((const void *)chunk_attn_kernel<false, true>, Roles<true>::kThreads) ||
        !add((const void *)chunk_attn_kernel<true, true>, Roles<true>::kThreads))
        return 0;
    return g_clusters[dev] = least;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 f = known.load(std::memory_order_relaxed);
    if (!f) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !fn)
            return nullptr;
        f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        known.store(f, std::memory_order_relaxed);
    }
    return f;
}

// q as rows of 512 values, boxes of 64 columns by R rows in the MMA's 128-byte swizzle.
bool make_q_map(CUtensorMap *map, const void *q, int64_t nrows, int R) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)nrows};
    cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    cuuint32_t box[2] = {64, (cuuint32_t)R};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The workspace's rows [b * (wrows + crows)][512] as chunks of 64 columns: boxes of `rows` rows of `chunks` chunks, each
// chunk's rows together, in the MMA's 128-byte swizzle.
bool make_rows_map(CUtensorMap *map, const void *rows, int64_t n, int box_rows, int box_chunks) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {64, (cuuint64_t)n, 8};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)box_chunks};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(rows), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
    int R, nqt, parts, clusters;
    int64_t whole, units;      // units that are not in parts, and with the parts of the others
    bool wide;
    int wrows, crows;          // wide: rows of a sequence in the workspace
    void no_rows() {
        wide = false;
        wrows = crows = 0;
    }
};

// Query rows a CTA: the fewest that hold a sequence's queries in one unit.
// Rows widened once in a pass of their own (wide) when several units of a sequence read them, and they take no more than
// 2 GB.
// Parts of a unit: with fewer units than clusters, the number of least estimated time, in tiles: rounds of units, each its
// tiles and two for its ends, and from two parts on 1 + 0.02 k for the merge (at 3 + 0.05 k units of four tiles stayed whole: one
// sequence of 448 rows and 128 heads 18.1 us instead of 15.1; all else was the same).  With more, those of a last round
// that would leave half of the clusters or more without work are cut into as many parts as there are clusters for, where
// that saves more than the merge takes (8 tiles' time).
bool plan(int b, int m, int h, int window, int ratio, int page, int max_pages, Plan &pl) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const int g = max_clusters(dev);
    if (g <= 0) return false;
    const int64_t nr = (int64_t)m * h;
    pl.R = nr <= 32 ? 16 : nr <= 64 ? 32 : 64;
    pl.nqt = (int)((nr + 2 * pl.R - 1) / (2 * pl.R));
    const int64_t units = (int64_t)b * pl.nqt, cap = std::min<int64_t>((int64_t)max_pages * page, kMaxRows);
    // (a ring holds every position that the chunk sees, and the block table holds the ring)
    const int64_t wr = (window ? std::min<int64_t>((int64_t)window + m - 1, cap) : cap) + BN, cr = ratio ? cap + BN : 0;
    pl.wide = pl.nqt >= kWideTiles && (wr + cr) * b * (D * 2) <= (int64_t)2 << 30;
    pl.wrows = pl.wide ? (int)wr : 0;
    pl.crows = pl.wide ? (int)cr : 0;
    // rows that a unit can have at most, for all that the host knows
    const int64_t span = (2 * pl.R + h - 2) / h;
    int64_t most = window ? std::min<int64_t>(cap, (int64_t)window + span) : cap;
    if (ratio) most = std::min(cap, most + cap);
    const int64_t tiles = std::max<int64_t>(1, (most + BN - 1) / BN);
    pl.parts = 1;
    pl.whole = units;
    if (units <= g) {
        double least = 1e30;
        for (int k = 1; k <= kMaxParts && k <= tiles; ++k) {
            const double rounds = (double)((units * k + g - 1) / g);
            const double cost = rounds * ((double)((tiles + k - 1) / k) + 2.0) + (k > 1 ? 1.0 + 0.02 * k : 0.0);
            if (cost < least) {
                least = cost;
                pl.parts = k;
            }
        }
        if (pl.parts > 1) pl.whole = 0;
    } else if (units < 8 * (int64_t)g && units % g != 0) {
        const int64_t rest = units % g, k = std::min<int64_t>({g / rest, tiles, kMaxParts});
        if (k >= 2 && tiles - (tiles + k - 1) / k >= 8) {
            pl.parts = (int)k;
            pl.whole = units - rest;
        }
    }
    pl.units = pl.whole + (units - pl.whole) * pl.parts;
    pl.clusters = (int)std::min<int64_t>(pl.units, g);
    return pl.units < UINT32_MAX / 2;
}

size_t rows_bytes(const Plan &pl, int b) { return (size_t)b * (size_t)(pl.wrows + pl.crows) * (D * 2); }
size_t workspace_bytes(const Plan &pl, int b) {
    return rows_bytes(pl, b) + (size_t)(pl.units - pl.whole) * (pl.parts > 1 ? 1 : 0) * (D + 2) * (2 * pl.R) * sizeof(float);
}

}  // namespace chunk

void set_test_stall_chunk(bool on) { chunk::g_test_stall.store(on ? 1 : 0, std::memory_order_relaxed); }

size_t chunk_attn_fp8_workspace_bytes(int b, int m, int h, int window, int ratio, int page, int max_pages) {
    chunk::Plan pl;
    if ((int64_t)b * m == 0 || !chunk::plan(b, m, h, window, ratio, page, max_pages, pl)) return 0;
    return chunk::workspace_bytes(pl, b);
}

int launch_chunk_attn_fp8(const chunk::Args &a, cudaStream_t stream) {
    using namespace chunk;
    Plan pl;
    if (!plan(a.b, a.m, a.h, a.window, a.ratio, a.page, a.max_pages, pl)) return launch_failed();
    // with lens, a chunk as long as m may see more positions than the table has rows: the workspace would not hold them
    if (a.ring && (int64_t)a.window + a.m - 1 > (int64_t)a.max_pages * a.page) pl.no_rows();
    const size_t need = workspace_bytes(pl, a.b);
    if (a.workspace_bytes < need || (need && !a.workspace)) return DS_EWORKSPACE;
    char *ws = static_cast<char *>(a.workspace);
    auto over = [](int64_t v) { return Divisor((uint32_t)std::max<int64_t>(v, 1)); };
    Params p{a, over(a.h), over(a.page), over(a.ring), over(a.b), over(pl.parts), over(a.ratio), pl.R, pl.nqt, (uint32_t)pl.units,
             (uint32_t)pl.whole, over(pl.clusters), std::min<int64_t>((int64_t)a.max_pages * a.page, kMaxRows), a.scale * kLog2e,
             reinterpret_cast<float *>(ws + (pl.wide ? rows_bytes(pl, a.b) : 0)),
             pl.wide ? reinterpret_cast<uint16_t *>(ws) : nullptr, pl.wrows, pl.crows, g_test_stall.load(std::memory_order_relaxed)};
    if (a.pages == 0) {       // rows without a slot are read from slot 0, for nothing: there it is q's first row
        p.a.codes = reinterpret_cast<const uint8_t *>(a.q);
        p.a.exps = reinterpret_cast<const int8_t *>(a.q);
    }
    CUtensorMap qmap, kmap, vmap;
    if (!make_q_map(&qmap, a.q, (int64_t)a.b * a.m * a.h, pl.R)) return DS_ECUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    // programmatic dependent launches: the set-up overlaps the previous kernel on the stream
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (pl.wide) {
        const int64_t n = (int64_t)a.b * (pl.wrows + pl.crows);
        if (!make_rows_map(&kmap, ws, n, HR, 4) || !make_rows_map(&vmap, ws, n, BN, 2)) return DS_ECUDA;
        cfg.gridDim = dim3((unsigned)((pl.wrows + kRowsBlock - 1) / kRowsBlock + (pl.crows + kRowsBlock - 1) / kRowsBlock), (unsigned)a.b, 1);
        cfg.blockDim = dim3(256, 1, 1);
        if (cudaLaunchKernelEx(&cfg, chunk_rows_kernel, p) != cudaSuccess) return launch_failed();
    } else {
        kmap = vmap = qmap;
    }
    const bool split = pl.parts > 1;
    auto kernel = split ? (pl.wide ? chunk_attn_kernel<true, true> : chunk_attn_kernel<true, false>)
                        : (pl.wide ? chunk_attn_kernel<false, true> : chunk_attn_kernel<false, false>);
    cfg.gridDim = dim3((unsigned)(2 * pl.clusters), 1, 1);
    cfg.blockDim = dim3((unsigned)(pl.wide ? Roles<true>::kThreads : Roles<false>::kThreads), 1, 1);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    if (cudaLaunchKernelEx(&cfg, kernel, qmap, kmap, vmap, p) != cudaSuccess) return launch_failed();
    if (split) {
        auto merge = pl.parts > kManyParts ? chunk_merge_kernel<16> : chunk_merge_kernel<4>;
        cfg.gridDim = dim3((unsigned)((pl.units - pl.whole) / pl.parts), (unsigned)(2 * pl.R), 1);
        cfg.blockDim = dim3(128, 1, 1);
        cfg.dynamicSmemBytes = 0;
        if (cudaLaunchKernelEx(&cfg, merge, p) != cudaSuccess) return launch_failed();
    }
    return DS_OK;
}

}  // namespace dsattn
