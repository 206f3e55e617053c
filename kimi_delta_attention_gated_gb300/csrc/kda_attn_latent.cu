// kda_attn_latent.cu -- attention over the paged latent cache, in the latent's space.
//
//   o[t, h] = sum_j softmax_j(scale * q[t, h] . row_j) row_j[0:512],   j < seen_t,
//
// rows of 576 channels, the same for all heads.  A sequence's query rows (its tokens times the
// heads) are taken in tiles of up to 64, which share one pass over the cache.
//
// Products, on tcgen05, 64 cached tokens a step:
//   S  [query rows (M 64) x tokens (64)]   = Q C^T,   K = 576; both K-major,
//   O^T[channels (4 x M 128) x query rows] += C^T P^T, K = 64: the same bytes of C, read MN-major.
// O stands transposed because 64 rows of 512 channels fill only half of TMEM's lanes the other way,
// and because its products' second operand, P^T, then is what a softmax thread writes: a
// row's 64 weights are one swizzled 128-byte line.
//
// Shared memory is what limits a tile to 64 rows and the ring to two and a half steps of the cache: of
// a query's nine blocks of 64 channels five or three lie there, and the other four or six in TMEM, which a
// product of 64 rows may read its first operand from and has room beside O^T and two steps' scores
// (8 sequences of 60000 tokens, 96 heads: 151 us with all in shared memory, 140 and 134).  The cache arrives by TMA in a ring of
// 128-channel units of 16 KB (the shared channels in one of their own of 8 KB), and a unit is free again
// when the one product of O^T that reads it is through.  (Units of 32 KB, half the waits: 145 us.)  A step's scores
// are formed while the softmax works on the last step's.  The softmax's reference moves only where a row's maximum
// rises by more than 2^kSlack, since moving it means rescaling O^T in TMEM.
//
// Work split.  All steps of all units (a sequence's groups of G tiles, each tile on a CTA of
// its own, so that the G read the same tokens at about the same time and all but one find them in
// L2) are numbered in one line, kPad places before each unit standing for what it costs beside its steps; the
// line is cut into equal pieces.  Units that more than one CTA took leave their sums in a
// workspace, and attn_latent_join_kernel adds them in their order, so results do not depend on timing.
// Where the lengths allow it, units go whole to the piece that they begin in; where the table's width already says so
// (plan_of), the second launch falls away.  A table that is wider than the sequences need keeps it: 32 heads, 64 sequences of
// 5 tokens 9.1 and 13.6 us, 128 of about 1000 34.6 and 39.5, one of 1000 14.7 and 15.3.
// Every unit of a sequence has places for all of the sequence's steps.  In steps and drafts that is what it takes; of a
// fresh prompt's piece, though, the early tokens see little, and the pieces are not equal work: with 4096 fresh rows of 16 heads
// the busiest CTA has 1.9 times the mean (510 us, of which operations need 151), with 512 rows behind 4096 1.1 (98 and 40).
//
// What bounds it.  Up to 64 heads and long contexts: HBM.  8 sequences of 60000 tokens: 96 us with 16 heads, 104 with 64,
// 5.8 and 5.3 TB/s of 6.7 that a copy reaches.  96 and 128 heads are two tiles and twice the products: 134 and
// 143 us, 2200 and 2300 cycles a step of which its operands take 1900 (S reads 72 KB of C and up to 40 KB of Q through
// shared memory's 128 bytes a cycle, O^T 64 KB of C and P four times).  Neither that nor the tensor core binds by itself: with 16 of
// the 36 score products left out a step gains 5%; a ring place less costs as much (152 us with 128 heads; weights in two
// buffers instead gain nothing).  Short calls are launches and latencies: one sequence of 1000 tokens 14 us, of which the
// set-up takes 3, the first data 2, the output 3 and the joining launch 5; 128 of about 1000 tokens, 32 heads, 35 us, HBM's
// 22 between such a beginning and end.  An item's end in the middle of a CTA's run costs about 4 steps (kPad).
#include <cuda.h>

#include <climits>

#include <algorithm>
#include <cstring>

#include "kda_chunk_common.cuh"
#include "kda_latent.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kStep = 64;               // cached tokens of a step
constexpr int kTileRows = 64;           // query rows of a tile at most
constexpr int kSoftWarps = 4, kScoreWarp = 4, kValueWarp = 5, kLoadWarp = 6, kQueryWarp = 8;
constexpr int kQueryWarps = 4;
constexpr int kThreads = (kQueryWarp + kQueryWarps) * 32;
constexpr int kSlots = 4;               // work items under way
// A unit's own cost in steps (its queries' copy, the first data, its output).  By 0, 2, 4 and 6: 37 sequences of 3 to 5000
// tokens, 1 to 6 rows, 16 heads 42.3, 30.1, 26.2, 25.7 us; 170 of up to 4036, 128 heads 144, 129, 126, 126; 167 of up to
// 737, 1 to 3 rows, 5 heads 36.6, 31.3, 31.9, 33.4.
constexpr int kPad = 4;
constexpr int kMostPieces = 160, kMostSteps = 1 << 19;
// What cutting costs in steps at most (the sums' way through L2, their joining): units stay whole where no piece gets that
// much more by it.  Cut and whole: 64 sequences of 1000 tokens, 4 rows, 32 heads 47.4, 38.7 us; 256 sequences of about 1000,
// 64 heads 81.6, 74.5, 128 heads (more by 16 steps) 110, 114; 180 of 200 to 400 tokens, 16 heads (by 10) 27.0, 31.4.
constexpr int kCutCost = 12;
constexpr int kMaxShare = 8;            // tiles of a unit at most
constexpr double kIdle = 0.08;
constexpr int kMaxUnits = 12;            // ring places of units at most
constexpr uint32_t kShared = 2;         // and of the shared channels
constexpr uint32_t kUnitBytes = kStep * 256, kSharedBytes = kStep * 128;
constexpr uint32_t kTmemO = 2 * kStep;   // TMEM columns: scores of two steps, O^T, then queries
constexpr float kSlack = 8.f;           // log2: how far a score may exceed the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNaN = __builtin_nanf("");
constexpr int kMaxSmem = 232448;        // all that a CTA may have, so that nothing else on its SM wants TMEM
constexpr uint32_t kLastPolls = 256;    // for copies after a failure: a millisecond

__device__ int g_attn_latent_timeouts = 0;

struct Plan {
    int hp, tk;       // heads and tokens of a tile: hp * tk rows
    int parts;        // tiles that share a token's heads
    // Two ways to split, of which the lengths decide (without cuts both are the first).
    int G[2];         // tiles of a unit
    int pieces[2];    // of the line
    int units_one[2];  // units of a sequence with one token
    int ctas;
    int cut;          // units may be cut; else piece i is the i-th unit
    int by_unit;      // the joining launch goes by units, else by pieces
    int64_t most_places;  // tiles' places in the call's units at most
    int n;            // rows of a tile as the products' N: hp * tk up to a multiple of 16
    int q_rows;       // and as they lie in shared memory: up to a multiple of 8
    int q_units;      // of queries in shared memory: attn_latent_kernel's QU
    int units;        // ring places
    uint32_t at_p, at_units, at_shared, at_bars;  // shared memory
};

struct Args {
    AttnLatentParams p;
    Plan plan;
};

// One tile's share of a unit's steps.
struct Item {
    int found;
    int t0, tokens;       // rows of the call, [t0, t0 + tokens)
    int head0;
    int seen0;            // tokens that the first row sees (<= 0: none); each further one a token more
    int seq;
    int s0, s1;           // steps; s0 == s1: the tile sees nothing
    int64_t part;         // where its sums go in the workspace, or -1: written to o
    int bad;              // a page number out of range
};

struct Bars {
    uint64_t o_free, p_ready, s_free[2];  // arrivals: the softmax's warps
    uint64_t i_empty[kSlots];             // and the products' threads, and the queries' warps
    uint64_t qt_full;                     // the queries' warps
    uint64_t q_full, q_empty, p_free, drain[2], s_full[2], i_full[kSlots];  // one
    uint64_t u_full[kMaxUnits], u_empty[kMaxUnits], r_full[kShared], r_empty[kShared];
    Item slots[kSlots];
    union {
        struct {
            int64_t row_at[kTileRows];  // a row's place in o, or -1
            float factor[kTileRows];
        };
        int load[kMostPieces];          // while the line is measured: steps of the units that begin in a piece
    };
    int64_t scan[kThreads / 32][4];
    int64_t start_begin, start_unit;
    int start_seq;
    uint32_t tmem;
    int abort;                   // a bounded wait gave up
    uint32_t odd;                // the last item (from 1) with a cleared row that some of its tokens see
};

__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 lanes of 64 columns: the lower half of the warp's threads reads columns 0 to 31, the upper half the
// same lanes' columns 32 to 63.
__device__ __forceinline__ void tmem_ld_halves(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], 32;"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}
// The same for a store: the lower half of the warp's threads writes 16 lanes' columns 0 to 31, the upper half the
// same lanes' columns 32 to 63.
__device__ __forceinline__ void tmem_st_halves(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x32.b32 [%0], 32, {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
}
// Waits for the loads issued so far; naming the registers keeps their uses behind the wait.
template <int N>
__device__ __forceinline__ void wait_ld(float *r) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < N; i += 8)
        asm volatile("" : "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]),
                     "+f"(r[i + 6]), "+f"(r[i + 7]));
}
__device__ __forceinline__ void tmem_ld16f(uint32_t taddr, float *r) {
    uint32_t u[16];
    tmem_ld16(taddr, u);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(u[i]);
}
// 16 lanes of 16 columns: of each 8 columns a thread has 2 (lane % 4) and the next, of lane / 4 (registers 0, 1) and of
// the lane eight further (2, 3), which is how the matrices of stmatrix lie.
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, float *r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr));
}
// Four 8 x 8 matrices, turned: a row of memory, 16 bytes at the address from lane 8 * matrix + row, is a column.
__device__ __forceinline__ void st_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// Stores without a branch.
__device__ __forceinline__ void store_if(bool x, void *p, float v) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(p), "f"(v),
                 "r"((uint32_t)x)
                 : "memory");
}
// A 128-byte-swizzled operand's descriptor from its low word (address / 16 and leading offset);
// the row groups are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}
// mbar_try_wait, mbar_arrive_expect_tx and a copy, the barrier by its shared-memory address.
__device__ __forceinline__ bool try_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void expect_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_at(uint32_t dst, const void *tmap, uint32_t bar, int row, int block) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(0), "r"(row), "r"(block), "r"(bar)
        : "memory");
}
// A barrier of the softmax's warps that also says whether any of their threads has `x`.
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

// ---------------------------------------------------------------------------
// the line

__device__ __forceinline__ int tokens_of(const LatentCache &c, int n) {
    const int64_t room = (int64_t)c.max_blocks << c.p_shift;
    return (int)max((int64_t)0, min((int64_t)__ldg(c.lens + n), room));
}
__host__ __device__ __forceinline__ int steps_of(int tokens) { return (int)(((int64_t)tokens + kStep - 1) / kStep); }
// Units of a sequence with nq rows in the call (tiles stay below 2^31: 2^24 rows, 64 tiles of a token).
__host__ __device__ __forceinline__ int units_of(const Plan &pl, int way, int nq) {
    if (nq <= 1) return nq * pl.units_one[way];
    const uint32_t tiles = ((uint32_t)nq + pl.tk - 1) / pl.tk * pl.parts;
    return (int)((tiles + pl.G[way] - 1) / pl.G[way]);
}
// Its units, and their places on the line.
__device__ __forceinline__ int units_of(const Args &a, int way, int n) {
    int64_t t0;
    int nq;
    call_rows(a.p.cu_seqlens, a.p.tokens, n, t0, nq);
    return units_of(a.plan, way, nq);
}
// Places of a unit beside its own cost (one without steps has a place too: its rows are written there): the whole sequence's,
// also where its tokens see less.
__device__ __forceinline__ int line_steps(int len) { return max(1, steps_of(len)); }
__device__ __forceinline__ int seq_steps(const Args &a, int n) { return line_steps(tokens_of(a.p.c, n)); }

// Every thread's share [first, last) of the sequences measured: the steps and units of all sequences, and
// of those before the share.
struct Line {
    int64_t total, total_units, mine, units;
    int first, last;
    int way;
};
template <int THREADS>
__device__ __forceinline__ Line measure_line(const Args &a, int64_t (*scan)[4]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.p.c.N, per = (N + THREADS - 1) / THREADS;
    Line l;
    l.first = min(tid * per, N);
    l.last = min(l.first + per, N);
    const bool ways = a.plan.G[0] != a.plan.G[1];
    int64_t x[2] = {}, y[2] = {};
    for (int n = l.first; n < l.last; ++n) {
        const int64_t steps = seq_steps(a, n);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (w == 1 && !ways) break;
            const int64_t u = units_of(a, w, n);
            y[w] += u;
            x[w] += u * steps;
        }
    }
    const int64_t own[2] = {x[0], x[1]}, own_units[2] = {y[0], y[1]};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (w == 1 && !ways) break;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t dx = __shfl_up_sync(0xffffffffu, x[w], o), dy = __shfl_up_sync(0xffffffffu, y[w], o);
            if (lane >= o) x[w] += dx, y[w] += dy;
        }
        if (lane == 31) scan[warp][2 * w] = x[w], scan[warp][2 * w + 1] = y[w];
    }
    __syncthreads();
    l.way = 0;
    if (ways) {  // the second way, unless it leaves too many CTAs without a tile: see share_of
        int64_t t[2] = {};
        for (int w = 0; w < THREADS / 32; ++w) t[0] += scan[w][0], t[1] += scan[w][2];
        l.way = (double)t[1] * a.plan.pieces[0] <= (1. + kIdle) * (double)t[0] * a.plan.pieces[1];
    }
    l.mine = l.way ? x[1] - own[1] : x[0] - own[0];
    l.units = l.way ? y[1] - own_units[1] : y[0] - own_units[0];
    l.total = l.total_units = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        const int64_t dx = scan[w][2 * l.way], dy = scan[w][2 * l.way + 1];
        if (w < warp) l.mine += dx, l.units += dy;
        l.total += dx;
        l.total_units += dy;
    }
    return l;
}

// A tile's rows and what they see.
struct Tile {
    int t0, tokens, head0, seen0, steps;
};
__device__ __forceinline__ Tile tile_of(const Plan &pl, int64_t t0, int nq, int len, int r) {
    const int of = r / pl.parts, i0 = of * pl.tk;
    Tile t;
    t.head0 = (r - of * pl.parts) * pl.hp;
    t.tokens = max(0, min(pl.tk, nq - i0));
    t.t0 = (int)t0 + i0;
    t.seen0 = len - nq + i0 + 1;
    t.steps = t.tokens > 0 ? steps_of(max(0, t.seen0 + t.tokens - 1)) : 0;
    return t;
}
// What a part leaves in the workspace (two a CTA): O as [128-channel block][row / 4][channel][row % 4], the rows' references
// and their sums.
__host__ __device__ __forceinline__ int64_t part_floats(const Plan &pl) { return (int64_t)pl.n * (kLatent + 2); }

// What the joining launch has to know of a tile that begins in a piece and goes on behind it.
struct __align__(16) JoinWord {
    int t0, place, first, last;  // its first row; its first head and its rows' tokens << 16; the pieces of its
                                 // first and its last step
};
// These words lie behind the parts: with by_unit one for each of a unit's G tiles, else one for each CTA, then one
// with the number of units or pieces and with G.  first == last: nothing to join.
__host__ __device__ __forceinline__ int64_t words_of(const Plan &pl) { return pl.by_unit ? pl.most_places : pl.ctas; }
__device__ __forceinline__ int4 *join_words(const Args &a) {
    return reinterpret_cast<int4 *>(a.p.ws + (int64_t)a.plan.ctas * 2 * part_floats(a.plan));
}

// Goes through the work items of one tile place `g` of a piece.
struct Walk {
    int way, G;
    bool whole;                // units go whole to the piece that they begin in
    int64_t L0, L1, S, begin;  // the piece, the next unit's place on the line (without cuts: units)
    int n, u, units, nq, len;  // the next unit: its sequence, and number there
    int64_t t0;
    int pad;
    bool open;
    int64_t unit;              // the next unit's number in the call
    JoinWord join;             // of the last item that begins and is cut
    __device__ void look(const Args &a) {  // at sequence n, or the next one with rows
        for (;; ++n) {
            if (n >= a.p.c.N) return;
            call_rows(a.p.cu_seqlens, a.p.tokens, n, t0, nq);
            if (nq > 0) break;
        }
        len = tokens_of(a.p.c, n);
        units = units_of(a.plan, way, nq);
        open = true;
    }
    __device__ void start(const Args &a, int split, bool uncut, int64_t l0, int64_t l1, int64_t s, int own, int seq, int64_t seq_begin, int64_t seq_unit) {
        way = split;
        whole = uncut;
        G = a.plan.G[way];
        L0 = l0;
        L1 = l1;
        S = s;
        pad = own;
        open = false;
        join.t0 = join.place = join.first = join.last = 0;
        n = seq < 0 ? a.p.c.N : seq;
        if (n >= a.p.c.N) return;
        look(a);
        const int64_t per = a.plan.cut ? line_steps(len) + pad : 1;
        u = (int)((l0 - seq_begin) / per);
        begin = seq_begin + u * per;
        unit = seq_unit + u;
    }
    // (words: by this thread the joining launch's words by unit are written)
    __device__ Item next(const Args &a, int piece, int g, bool words) {
        const Plan &pl = a.plan;
        Item it = {};
        while (n < a.p.c.N && begin < L1) {
            if (!open) look(a);
            if (n >= a.p.c.N) break;
            const int64_t first = begin + pad, at = begin;
            const Tile t = tile_of(pl, t0, nq, len, u * G + g);
            it.seq = n;
            begin += pl.cut ? line_steps(len) + pad : 1;
            const int64_t number = unit++;
            if (++u == units) {
                ++n;
                u = 0;
                open = false;
            }
            // (a cu_seqlens that does not ascend may have more units than there is room for)
            const int64_t starts = at + (t.steps && !whole ? pad : 0);
            if (words && pl.cut && pl.by_unit && number * G + g < pl.most_places && starts >= L0 && starts < L1) {
                const int last = t.steps && !whole ? (int)((first + t.steps - 1) / S) : piece;
                join_words(a)[number * G + g] = make_int4(t.t0, t.head0 | t.tokens << 16, piece, t.tokens ? last : piece);
            }
            if (t.tokens == 0) continue;
            it.t0 = t.t0;
            it.tokens = t.tokens;
            it.head0 = t.head0;
            it.seen0 = t.seen0;
            it.part = -1;
            if (whole || t.steps == 0) {
                if (at < L0) continue;  // the piece's before
                it.s0 = 0;
                it.s1 = t.steps;
            } else {
                it.s0 = (int)max(L0 - first, (int64_t)0);
                it.s1 = (int)min(L1 - first, (int64_t)t.steps);
                if (it.s0 >= it.s1) continue;
                if (it.s0 > 0 || it.s1 < t.steps)
                    it.part = (((int64_t)piece * G + g) * 2 + (it.s0 > 0 ? 0 : 1)) * part_floats(pl);
                if (it.s0 == 0 && it.s1 < t.steps) {
                    join.t0 = t.t0;
                    join.place = t.head0 | t.tokens << 16;
                    join.first = piece;
                    join.last = (int)((first + t.steps - 1) / S);
                }
            }
            it.found = 1;
            return it;
        }
        return it;
    }
};

// QU: of a query's four units of 128 channels, in shared memory; the others lie in TMEM, whose 512 columns are 128 of scores,
// 4 n of O^T and 64 a unit.
template <int QU>
__global__ void __launch_bounds__(kThreads, 1)
    attn_latent_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c,
                       const __grid_constant__ CUtensorMap map_r, const __grid_constant__ Args a) {
    const AttnLatentParams &p = a.p;
    const Plan &pl = a.plan;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm), sb16 = (sb & 0x3FFFF) >> 4;
    Bars &b = *reinterpret_cast<Bars *>(sm + pl.at_bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t q_rows = pl.hp * pl.tk;
    constexpr int kQBlocks = 2 * QU + 1;  // of 64 channels, in shared memory; the last: the shared channels
    volatile int *abort_flag = &b.abort;

    if (pl.cut) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    constexpr int kBars = offsetof(Bars, slots) / 8, kBarsSoft = offsetof(Bars, i_empty) / 8, kBarsItems = offsetof(Bars, qt_full) / 8;
    static_assert(kBars <= kThreads, "a thread for each barrier");
    if (threadIdx.x < kBars) {
        mbar_init(reinterpret_cast<uint64_t *>(&b) + threadIdx.x,
                  threadIdx.x < kBarsSoft    ? kSoftWarps
                  : threadIdx.x < kBarsItems ? kSoftWarps + 2 + kQueryWarps
                  : threadIdx.x == kBarsItems ? kQueryWarps
                                              : 1);
        fence_mbar_init();
    }
    if (threadIdx.x < kMostPieces) b.load[threadIdx.x] = 0;
    if (threadIdx.x == kThreads - 1) {
        b.abort = 0;
        b.odd = 0;
        b.start_seq = -1;
    }
    if (warp == kLoadWarp && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &map_q : lane == 1 ? &map_c : &map_r) : "memory");
    if (warp == kScoreWarp) {
        tmem_alloc(&b.tmem, 512);
        tmem_relinquish();
    }
    // What is above overlaps the end of the launch before; from here on its results are read.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == kLoadWarp && !pl.cut && !p.cu_seqlens) {
        // the length and the first pages on their way, while the rest is set up
        const int n = blockIdx.x / pl.G[0] / pl.units_one[0];
        int x, y = 0;
        asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(x) : "l"(p.c.lens + n));
        if (lane < p.c.max_blocks) asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(y) : "l"(p.c.block_table + (int64_t)n * p.c.max_blocks + lane));
        asm volatile("" ::"r"(x), "r"(y));
    }
    // The piece: places of the line, or without cuts units.
    int64_t L0, L1, S = 1;
    int pad = 0, way = 0, piece;
    bool whole = !pl.cut;
    int start_seq;
    int64_t start_begin, start_unit = 0, total_units = 0;
    if (!pl.cut && !p.cu_seqlens) {  // as many units in every sequence
        piece = blockIdx.x / pl.G[0];
        L0 = piece;
        L1 = piece + 1;
        start_seq = piece / pl.units_one[0];
        start_begin = (int64_t)start_seq * pl.units_one[0];
    } else {
        const Line line = measure_line<kThreads>(a, b.scan);  // (a barrier inside)
        way = line.way;
        piece = blockIdx.x / pl.G[way];
        L0 = piece;
        L1 = piece + 1;
        if (pl.cut) {
            pad = kPad;
            const int64_t places = line.total + pad * line.total_units;
            S = (places + pl.pieces[way] - 1) / pl.pieces[way];
            L0 = piece * S;
            L1 = min(L0 + S, places);
            total_units = line.total_units;
        }
        // With a few units a piece it may take less time to leave them whole.
        const bool look = pl.cut && 2 * total_units > pl.pieces[way] && total_units <= 8 * pl.pieces[way] && S < kMostSteps &&
                          pl.pieces[way] <= kMostPieces;
        int64_t at = pl.cut ? line.mine + pad * line.units : line.units, units = line.units;
        for (int n = line.first; n < line.last; ++n) {
            const int64_t more = (int64_t)units_of(a, way, n) * (pl.cut ? seq_steps(a, n) + pad : 1);
            if (L0 >= at && L0 < at + more && L0 < L1) {
                b.start_seq = n;
                b.start_begin = at;
                b.start_unit = units;
            }
            if (look) {
                // (one with many units is cut: they are too many to look at by one thread)
                const int each = seq_steps(a, n) + pad, most = more > 8 * (int64_t)each ? 2 * kMostSteps : min(each, 2 * kMostSteps);
                for (int64_t x = at; x < at + (most == each ? more : min(more, (int64_t)1)); x += each) atomicAdd(&b.load[x / S], most);
            }
            at += more;
            units += units_of(a, way, n);
        }
        if (look) {
            __syncthreads();
            int most = 0;
            for (int i = lane; i < pl.pieces[way]; i += 32) most = max(most, b.load[i]);
            whole = __reduce_max_sync(0xffffffffu, most) <= S + min(kCutCost, 4 + pl.n / 4);
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = b.tmem;
    if (pl.cut || p.cu_seqlens) {
        start_seq = b.start_seq;
        start_begin = b.start_begin;
        start_unit = b.start_unit;
    }
    const int G = pl.G[way], g = blockIdx.x - piece * G;
    auto last_words = [&](const Walk &w) {
        if (!pl.by_unit) join_words(a)[blockIdx.x] = *reinterpret_cast<const int4 *>(&w.join);
        if (blockIdx.x == 0)
            join_words(a)[words_of(pl)] = make_int4(pl.by_unit ? (int)min(total_units, pl.most_places / G) : pl.pieces[way], G, 0, 0);
    };
    auto wait_for = [&](uint64_t *bar, uint32_t parity, uint32_t polls) {
        for (uint32_t i = 0; i < polls; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) break;
        }
        *abort_flag = 1;
        return false;
    };
    auto wait_at = [&](uint32_t bar, uint32_t parity) {
        for (uint32_t i = 0; i < kAttnPolls; ++i) {
            if (try_at(bar, parity)) return true;
            if (*abort_flag) break;
        }
        *abort_flag = 1;
        return false;
    };
    // All lanes of a warp go on or stop together.
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar, parity, kAttnPolls)) != 0; };

    if (warp >= kLoadWarp && warp < kQueryWarp) {
        // ---- work items, and the copies of the cache, from a thread of each of two warps: the first has a step's
        // shared channels and units 0 and 1, the second the other two.  A thread by itself issues an instruction
        // every five cycles or so: all copies of a step took one thread 2200 cycles, or with the warp's votes about
        // each wait 2900, and either was the bound.
        if (elect_one()) {
            const int half = warp - kLoadWarp;
            Walk w;
            w.start(a, way, whole, L0, L1, S, pad, start_seq, start_begin, start_unit);
            uint32_t us = 0, up = 1;           // ring place of the step's first unit, and the parity of the wait for it (a
                                               // barrier's phase before its first counts as over)
            uint32_t rs = 0, rp = 1, steps = 0;
            bool ok = true;
            const uint32_t at_full = smem_u32(b.u_full), at_empty = smem_u32(b.u_empty), to_units = sb + pl.at_units;
            const int sub = min(kStep, p.c.P), per_step = kStep / sub;              // rows of a copy
            const int in_page = p.c.p_shift - (sub == 16 ? 4 : sub == 32 ? 5 : 6);  // log2 of a page's copies
            const int page_mask = (1 << in_page) - 1, sub_shift = p.c.p_shift - in_page;
            // Page numbers of a step's copies, looked up a step ahead (an item's first while the one before is
            // copied).  kNone: behind what the tile needs.
            constexpr int kNone = INT_MIN;
            struct Pages {
                int at[4];
            };
            auto look_up = [&](const int32_t *table, int need, int s) {
                Pages q;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int i = s * per_step + j;
                    q.at[j] = kNone;
                    if (j < per_step && (uint32_t)i < (uint32_t)need) {
                        const int page = __ldg(table + (i >> in_page));
                        q.at[j] = (uint32_t)page < (uint32_t)p.c.n_pages ? page : -1;
                    }
                }
                return q;
            };
            auto table_of = [&](const Item &it) { return p.c.block_table + (int64_t)it.seq * p.c.max_blocks; };
            // Copies that the tile needs, from the sequence's first.
            auto need_of = [&](const Item &it) {
                return it.found && it.s1 > it.s0 ? (min(it.seen0 + it.tokens - 1, it.s1 * kStep) + sub - 1) >> sub_shift : 0;
            };
            Item ahead = w.next(a, piece, g, half == 0);
            Pages first = look_up(table_of(ahead), need_of(ahead), ahead.s0);
            for (uint32_t k = 0; ok; ++k) {
                const Item it = ahead;
                Pages pages = first;
                const int slot = k % kSlots;
                if (half == 0) {
                    if (k >= kSlots) ok = wait_for(b.i_empty + slot, (k / kSlots - 1) & 1, kAttnPolls);
                    if (!ok) break;
                    b.slots[slot] = it;
                    mbar_arrive(b.i_full + slot);
                }
                if (!it.found) break;
                ahead = w.next(a, piece, g, half == 0);
                first = look_up(table_of(ahead), need_of(ahead), ahead.s0);
                const int32_t *table = table_of(it);
                const int need = need_of(it);
                for (int s = it.s0; s < it.s1 && ok; ++s, ++steps) {
                    int at[4], bytes = 0;  // rows of the cache, -1: nothing to copy; of a block of 64 channels
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int page = pages.at[j];
                        at[j] = page < 0 ? -1 : (page << p.c.p_shift) + (((s * per_step + j) & page_mask) << sub_shift);
                        bytes += page < 0 ? 0 : 128 << sub_shift;
                        if (page < 0 && page != kNone && half == 0) *(volatile int *)&b.slots[slot].bad = 1;
                    }
                    pages = look_up(table, need, s + 1);
                    if (half == 0) {  // (the shared channels first: their scores come first)
                        ok = wait_for(b.r_empty + rs, rp, kAttnPolls);
                        if (!ok) break;
                        mbar_arrive_expect_tx(b.r_full + rs, bytes);
                        const uint32_t to = sb + pl.at_shared + rs * kSharedBytes;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (at[j] >= 0) tma_load_3d(to + j * sub * 128, &map_r, b.r_full + rs, 0, at[j], kLatent / 64);
                        if (++rs == kShared) rs = 0, rp ^= 1;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int m = 2 * half + i;
                        uint32_t place = us + m, parity = up;
                        if (place >= (uint32_t)pl.units) place -= pl.units, parity ^= 1;
                        ok = ok && wait_at(at_empty + place * 8, parity);
                        if (!ok) break;
                        const uint32_t full = at_full + place * 8, to = to_units + place * kUnitBytes;
                        expect_at(full, 2 * bytes);
                        if (per_step == 1) {  // both blocks of 64 channels at once
                            if (at[0] >= 0) tma_at(to, &map_c, full, at[0], 2 * m);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (at[j] >= 0) {
                                    tma_at(to + j * sub * 128, &map_r, full, at[j], 2 * m);
                                    tma_at(to + kSharedBytes + j * sub * 128, &map_r, full, at[j], 2 * m + 1);
                                }
                        }
                    }
                    if (!ok) break;
                    us += 4;
                    if (us >= (uint32_t)pl.units) us -= pl.units, up ^= 1;
                }
            }
            if (half == 0 && pl.cut && ok) last_words(w);
            // every copy lands before the CTA may end (after a failure within a step, those of that step may not have
            // been issued: their wait runs out)
            if (half == 0)
                for (uint32_t j = steps > kShared ? steps - kShared : 0; j < steps + !ok; ++j)
                    mbar_wait(b.r_full + j % kShared, (j / kShared) & 1, ok ? kAttnPolls : kLastPolls);
            const uint32_t fills = 4 * (steps + !ok), units = pl.units;
            for (uint32_t j = fills > units ? fills - units : 0; j < fills; ++j)
                if ((int)(j & 3) >> 1 == half) mbar_wait(b.u_full + j % units, (j / units) & 1, ok ? kAttnPolls : kLastPolls);
        }
        __syncwarp();
    } else if (warp == kScoreWarp || warp == kValueWarp) {
        // ---- products, the scores' and the values' each from one thread of a warp.  A look at a barrier
        // queues behind the products that its thread has issued, about 120 cycles in which the tensor core
        // idles; with two threads one's products run meanwhile.  (From one thread, with votes of its
        // warp, the same work took 4800 cycles a step, two threads then 2900.)
        const uint32_t k_major = (16u >> 4) << 16, mn_major = (kSharedBytes >> 4) << 16;
        const uint32_t u_at = sb16 + (pl.at_units >> 4);
        uint32_t blocks = 0, items = 0, us = 0, up = 0;  // steps and items with any so far; ring place and parity
        bool ok = true;
        if (elect_one()) {
            // The next item's steps: -1 at the end.
            int t0 = 0, head0 = 0;
            auto next_item = [&](uint32_t k) {
                ok = wait_for(b.i_full + k % kSlots, (k / kSlots) & 1, kAttnPolls);
                if (!ok) return -1;
                const Item &it = b.slots[k % kSlots];
                const int nt = it.found ? it.s1 - it.s0 : -1;
                t0 = it.t0;
                head0 = it.head0;
                mbar_arrive(b.i_empty + k % kSlots);
                return nt;
            };
            if (warp == kScoreWarp) {
                const uint32_t id = idesc_bf16(64, kStep, false, false, p.scale < 0.f);
                const uint32_t q_lo = sb16 | k_major, q_chunk = pl.q_rows * 128 >> 4, r_at = sb16 + (pl.at_shared >> 4);
                const uint32_t t_q = tb + kTmemO + 4 * pl.n;
                uint32_t rs = 0, rp = 0;
                for (uint32_t k = 0; ok; ++k) {
                    const int nt = next_item(k);
                    if (nt < 0) break;
                    if (nt == 0) continue;
                    // the queries, when the last item's scores are through (from this thread, so that the cache's
                    // copies do not wait for that: 6000 cycles at the border of two items)
                    if (items > 0) ok = wait_for(&b.q_empty, (items - 1) & 1, kAttnPolls);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&b.q_full, kQBlocks * q_rows * 128);
                    for (int x = 0; x < kQBlocks; ++x)
                        tma_load_3d(sb + x * pl.q_rows * 128, &map_q, &b.q_full, x == kQBlocks - 1 ? kLatent : x * 64, head0, t0);
                    ok = wait_for(&b.q_full, items & 1, p.polls);
                    if (!ok) mbar_wait(&b.q_full, items & 1, kAttnPolls);  // it still has to land before the CTA may end
                    ok = ok && wait_for(&b.qt_full, items & 1, kAttnPolls);
                    for (int s = 0; s < nt && ok; ++s, ++blocks) {
                        const uint32_t t_s = tb + (blocks & 1) * kStep;
                        if (blocks >= 2) ok = wait_for(b.s_free + (blocks & 1), ((blocks >> 1) - 1) & 1, kAttnPolls);
                        ok = ok && wait_for(b.r_full + rs, rp, p.polls);
                        if (!ok) break;
                        fence_after_sync();
                        {
                            const uint32_t lo = (r_at + rs * (kSharedBytes >> 4)) | k_major, ql = q_lo + (kQBlocks - 1) * q_chunk;
#pragma unroll
                            for (int x = 0; x < 4; ++x) mma_ss(t_s, desc_of(ql + 2 * x), desc_of(lo + 2 * x), id, x > 0);
                            mma_commit(b.r_empty + rs);
                            if (++rs == kShared) rs = 0, rp ^= 1;
                        }
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            ok = wait_for(b.u_full + us, up, p.polls);
                            if (!ok) break;
                            fence_after_sync();
                            const uint32_t lo = (u_at + us * (kUnitBytes >> 4)) | k_major, ql = q_lo + 2 * m * q_chunk;
#pragma unroll
                            for (int x = 0; x < 8; ++x) {
                                const uint64_t rows = desc_of(lo + (x >> 2) * (kSharedBytes >> 4) + 2 * (x & 3));
                                if (m < QU)
                                    mma_ss(t_s, desc_of(ql + (x >> 2) * q_chunk + 2 * (x & 3)), rows, id, 1);
                                else
                                    mma_ts(t_s, t_q + (m - QU) * 64 + 8 * x, rows, id, 1);
                            }
                            if (++us == (uint32_t)pl.units) us = 0, up ^= 1;
                        }
                        if (!ok) break;
                        mma_commit(b.s_full + (blocks & 1));
                    }
                    if (ok) mma_commit(&b.q_empty);
                    ++items;
                }
            } else {
                const uint32_t id = idesc_bf16(128, pl.n, true, false);
                const uint32_t p_lo = (sb16 + (pl.at_p >> 4)) | k_major, t_o = tb + kTmemO;
                for (uint32_t k = 0; ok; ++k) {
                    const int nt = next_item(k);
                    if (nt < 0) break;
                    if (nt == 0) continue;
                    if (items > 0) ok = wait_for(&b.o_free, (items - 1) & 1, kAttnPolls);  // the last item's output is read
                    for (int s = 0; s < nt && ok; ++s, ++blocks) {
                        ok = wait_for(&b.p_ready, blocks & 1, kAttnPolls);
                        if (!ok) break;
                        fence_after_sync();
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t lo = (u_at + us * (kUnitBytes >> 4)) | mn_major;
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                mma_ss(t_o + m * pl.n, desc_of(lo + x * (2048 >> 4)), desc_of(p_lo + 2 * x), id, s > 0 || x > 0);
                            mma_commit(b.u_empty + us);
                            if (++us == (uint32_t)pl.units) us = 0;
                        }
                        mma_commit(&b.p_free);
                    }
                    ++items;
                }
            }
            // nothing issued may still run, and no commit arrive, once the CTA has ended
            mma_commit(b.drain + (warp - kScoreWarp));
            mbar_wait(b.drain + (warp - kScoreWarp), 0, kAttnPolls);
        }
        __syncwarp();
    } else if (warp >= kQueryWarp) {
        // ---- the queries' other units into TMEM, where a 64-row operand's rows lie as the product leaves its own:
        // shared memory that holds more of the cache
        const int row = (warp - kQueryWarp) * 16 + (lane & 15), tok = row / pl.hp, head_in = row - tok * pl.hp;
        const uint32_t to = tb + ((uint32_t)((warp - kQueryWarp) * 32) << 16) + kTmemO + 4 * pl.n;
        uint32_t items = 0;
        for (uint32_t k = 0;; ++k) {
            if (!wait(b.i_full + k % kSlots, (k / kSlots) & 1)) break;
            const Item it = b.slots[k % kSlots];
            __syncwarp();
            if (lane == 0) mbar_arrive(b.i_empty + k % kSlots);
            if (!it.found) break;
            if (it.s0 == it.s1) continue;
            uint32_t r[4 - QU][32];  // of each unit this half of the warp's 64 channels
            const bool live = tok < it.tokens && it.head0 + head_in < p.H && row < (int)q_rows;
            const uint4 *q = reinterpret_cast<const uint4 *>(p.q + (int64_t)(it.t0 + tok) * p.q_stride + (int64_t)(it.head0 + head_in) * kRow +
                                                             QU * 128 + (lane >> 4) * 64);
#pragma unroll
            for (int j = 0; j < 4 - QU; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = live ? q[j * 16 + i] : make_uint4(0, 0, 0, 0);
                    r[j][4 * i] = v.x, r[j][4 * i + 1] = v.y, r[j][4 * i + 2] = v.z, r[j][4 * i + 3] = v.w;
                }
            if (items > 0 && !wait(&b.q_empty, (items - 1) & 1)) break;  // the last item's scores are through
            fence_after_sync();
#pragma unroll
            for (int j = 0; j < 4 - QU; ++j) tmem_st_halves(to + j * 64, r[j]);
            tmem_wait_st();
            fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.qt_full);
            ++items;
        }
        __syncwarp();
    } else {
        // ---- softmax, two threads per row (the M = 64 product leaves its rows in 16 of each warp's 32
        // lanes, which the lower half of a warp's threads read for 32 of the step's tokens and the
        // upper half for the others), and the output, a thread per channel
        constexpr int kHalf = kStep / 2;
        const int row = warp * 16 + (lane & 15), tok = row / pl.hp, head_in = row - tok * pl.hp;
        const int half = lane >> 4;
        const bool mine = half == 0;
        const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
        const float c = fabsf(p.scale) * kLog2e;
        uint32_t blocks = 0, items = 0;  // steps so far; items with any
        uint32_t us = 0;                 // ring place of the step's first unit
        uint32_t k = 0;
        bool ok = true;
        for (;; ++k) {
            // the four warps go on or stop together, since they wait for each other at barriers
            ok = wait(b.i_full + k % kSlots, (k / kSlots) & 1);
            if (soft_any(!ok)) {
                ok = false;
                break;
            }
            const Item it = b.slots[k % kSlots];
            if (!it.found) break;
            const int head = it.head0 + head_in, nt = it.s1 - it.s0;
            const bool live = tok < it.tokens && head < p.H && row < (int)q_rows;
            const int seen = it.seen0 + tok, most = it.seen0 + it.tokens - 1;  // of this row, of the tile
            float m = -INFINITY, l = 0.f;
            for (int s = 0; s < nt; ++s, ++blocks) {
                const int j0 = (it.s0 + s) * kStep;
                ok = ok && wait(b.s_full + (blocks & 1), (blocks >> 1) & 1);
                fence_after_sync();
                float x[kHalf];
                tmem_ld_halves(tb + lane_base + (blocks & 1) * kStep, x);
                wait_ld<kHalf>(x);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(b.s_free + (blocks & 1));
                if (j0 + kStep > it.seen0 || !live) {
                    const int lim = live ? seen - j0 - half * kHalf : 0;
#pragma unroll
                    for (int i = 0; i < kHalf; ++i)
                        if (i >= lim) x[i] = -INFINITY;
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int i = 4; i < kHalf; i += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[i + e]);
                mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const float mb = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], 16)) * c;
                const bool raise = mb > m + kSlack;  // (rows that are not live: never)
                if (soft_any(raise || !ok)) {
                    if (soft_any(!ok)) {
                        ok = false;
                        break;
                    }
                    const float f = raise ? ex2(m - mb) : 1.f;
                    if (raise) m = mb;
                    l *= f;
                    if (s > 0) {
                        ok = wait(&b.p_free, (blocks - 1) & 1);  // O holds all steps before
                        fence_after_sync();
                        if (mine) b.factor[row] = f;
                        if (soft_any(!ok)) {
                            ok = false;
                            break;
                        }
#pragma unroll 1
                        for (int r0 = 0; r0 < pl.n; r0 += 16) {
#pragma unroll 1
                            for (int q = 0; q < 4; ++q) {
                                float o[16];
                                const uint32_t at = tb + lane_base + kTmemO + q * pl.n + r0;
                                tmem_ld16f(at, o);
                                wait_ld<16>(o);
                                uint32_t u[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(o[i] * b.factor[r0 + i]);
                                tmem_st16(at, u);
                            }
                        }
                        tmem_wait_st();
                        fence_before_sync();
                        soft_sync();  // the factors may be written again
                    }
                }
                // The weights are rounded to bf16: a product's operands have one type, and the rows are bf16.  Off by 2^-8 each at
                // most, independently, which over 1000 tokens adds a quarter to the outputs' own rounding to bf16; the sum that divides
                // them is of the unrounded ones.
                const float mm = m == -INFINITY ? 0.f : m;
                float sum[2] = {0.f, 0.f};
                uint32_t w[kHalf / 2];
#pragma unroll
                for (int i = 0; i < kHalf; i += 2) {
                    const float e0 = ex2(fmaf(x[i], c, -mm)), e1 = ex2(fmaf(x[i + 1], c, -mm));
                    sum[0] += e0;
                    sum[1] += e1;
                    w[i / 2] = pack_bf16x2(e0, e1);
                }
                l += sum[0] + sum[1];
                // the last weights have to be multiplied before these take their place
                if (blocks > 0) ok = wait(&b.p_free, (blocks - 1) & 1);
                if (!ok) continue;  // (said to the other warps at the next barrier)
                if (row < pl.n) {
                    const uint32_t at = sb + pl.at_p + row * 128;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_shared_v4(at + (((4 * half + i) ^ (row & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
                if (j0 + kStep > it.seen0) {
                    // Tokens that not every row sees.  A weight of zero times what is not finite would not be
                    // zero: behind the tile's last token everything is cleared, and before it the rows
                    // that hold an infinity or a NaN, which those that see them get with the output.
                    for (int r = warp; r < kStep; r += kSoftWarps) {
                        if (j0 + r < it.seen0) continue;
                        uint32_t at[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // 16-byte pieces lane, lane + 32 of the 64
                            const int piece16 = lane + 32 * h, unit = piece16 >> 4;
                            uint32_t place = us + unit;
                            if (place >= (uint32_t)pl.units) place -= pl.units;
                            at[h] = sb + pl.at_units + place * kUnitBytes + ((piece16 >> 3) & 1) * kSharedBytes + r * 128 +
                                    (((piece16 & 7) ^ (r & 7)) << 4);
                        }
                        bool clear = j0 + r >= most;
                        if (!clear) {
                            bool odd = false;
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t v[4];
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at[h]));
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    odd |= (v[i] & 0x7F80u) == 0x7F80u || (v[i] & 0x7F800000u) == 0x7F800000u;
                            }
                            clear = __any_sync(0xffffffffu, odd);
                            if (clear && lane == 0) *(volatile uint32_t *)&b.odd = k + 1;
                        }
                        if (clear) {
                            st_shared_v4(at[0], 0, 0, 0, 0);
                            st_shared_v4(at[1], 0, 0, 0, 0);
                        }
                    }
                }
                us += 4;
                if (us >= (uint32_t)pl.units) us -= pl.units;
                fence_async_smem();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_ready);
            }
            // ---- output
            if (nt > 0) {
                ok = ok && wait(&b.p_free, (blocks - 1) & 1);
                fence_after_sync();
            }
            // All four warps come here, those that gave up too: a wait may run out in one warp and not in another, and
            // one that left by itself would keep the others at this barrier for ever.  (Also: the last item's places and
            // factors are read.)
            if (soft_any(!ok)) {
                ok = false;
                break;
            }
            l += __shfl_xor_sync(0xffffffffu, l, 16);  // of both halves of the tokens
            const bool bad = *(volatile int *)&b.slots[k % kSlots].bad != 0;
            if (bad) l = kNaN;
            if (*(volatile uint32_t *)&b.odd == k + 1) {
                // A channel that is infinite or NaN in a token that a row sees is NaN: the token's score is not finite either, and
                // where it is +inf or NaN the sum of weights is NaN, but where it is -inf the weight is 0, and 0 times that channel
                // NaN.  (As the products have it in steps that all rows see.)  A thread has a channel of each block, as in O^T.
                const int32_t *table = p.c.block_table + (int64_t)it.seq * p.c.max_blocks;
                const int j1 = min(most, it.s1 * kStep);
#pragma unroll 1
                for (int j = max(it.seen0, it.s0 * kStep); j < j1; ++j) {
                    const int page = __ldg(table + (j >> p.c.p_shift));
                    if ((uint32_t)page >= (uint32_t)p.c.n_pages) continue;  // (the rows are NaN)
                    const uint16_t *x = reinterpret_cast<const uint16_t *>(p.c.rows) +
                                        (((int64_t)page << p.c.p_shift) + (j & (p.c.P - 1))) * kRow + warp * 32 + lane;
#pragma unroll 1
                    for (int q = 0; q < 4; ++q) {
                        const bool odd = (__ldg(x + q * 128) & 0x7F80u) == 0x7F80u;
                        if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll 1
                        for (int r0 = 0; r0 < pl.n; r0 += 16) {
                            float o[16];
                            const uint32_t at = tb + lane_base + kTmemO + q * pl.n + r0;
                            tmem_ld16f(at, o);
                            wait_ld<16>(o);
                            uint32_t u[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                u[i] = __float_as_uint(odd && it.seen0 + (r0 + i) / pl.hp > j ? kNaN : o[i]);
                            tmem_st16(at, u);
                        }
                        tmem_wait_st();
                    }
                }
            }
            if (it.part >= 0) {
                // Sums of a part, four rows' values of a channel together, so that a warp's stores are
                // contiguous (a row's channels together, one store took 58 cycles, 12000 an item).
                float *ws = p.ws + it.part;
                if (mine && row < pl.n) {
                    ws[pl.n * kLatent + row] = m;
                    ws[pl.n * (kLatent + 1) + row] = l;
                }
                ws += (warp * 32 + lane) * 4;
#pragma unroll 1
                for (int at = 0; at < 4 * pl.n; at += 32) {
                    float o[32];
                    tmem_ld16f(tb + lane_base + kTmemO + at, o);
                    tmem_ld16f(tb + lane_base + kTmemO + at + 16, o + 16);
                    wait_ld<32>(o);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4 *>(ws + (int64_t)(at / 4 + e) * 512) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                }
            } else {
                if (mine) {
                    const int64_t out = live ? (int64_t)(it.t0 + tok) * p.H + head : -1;
                    b.row_at[row] = out;
                    b.factor[row] = l == 0.f ? 0.f : 1.f / l;
                    if (live && p.lse) p.lse[out] = l == 0.f ? -INFINITY : (log2f(l) + m) * kLn2;
                }
                soft_sync();
                if (p.o_bf16) {
                    // 16 rows and a warp's 32 channels at a time turned in 1 KB of the weights' room, 64 bytes of a row by
                    // four lanes.  (With a thread's channel of each row in stores of 2 bytes, 128 sequences of 1000 tokens
                    // took 39.4 us with 64 heads, now 38.0.)
                    const uint32_t room = sb + pl.at_p + warp * 1024;
                    const int at_row = ((lane >> 4) << 3) + (lane & 7), at_piece = (lane >> 3) & 1;  // for st_turned
                    __nv_bfloat16 *base = static_cast<__nv_bfloat16 *>(p.o) + warp * 32 + (lane & 3) * 8;
#pragma unroll 1
                    for (int r0 = 0; r0 < (int)q_rows; r0 += 16) {
                        float o[64], f[4];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            tmem_ld_quads(tb + lane_base + ((uint32_t)(i & 1) << 20) + kTmemO + (i >> 1) * pl.n + r0, o + 8 * i);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = b.factor[r0 + (i >> 1) * 8 + 2 * (lane & 3) + (i & 1)];
                        const int64_t to[2] = {b.row_at[r0 + (lane >> 2)], b.row_at[r0 + 8 + (lane >> 2)]};
                        wait_ld<64>(o);
                        if (nt == 0) {  // (then TMEM holds anything)
#pragma unroll
                            for (int i = 0; i < 64; ++i) o[i] = 0.f;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
#pragma unroll
                            for (int half = 0; half < 2; ++half) {  // 16 channels
                                const float *x = o + 16 * q + 8 * half;
                                st_turned(room + at_row * 64 + (((2 * half + at_piece) ^ ((at_row >> 1) & 3)) << 4),
                                          pack_bf16x2(x[0] * f[0], x[1] * f[1]), pack_bf16x2(x[2] * f[0], x[3] * f[1]),
                                          pack_bf16x2(x[4] * f[2], x[5] * f[3]), pack_bf16x2(x[6] * f[2], x[7] * f[3]));
                            }
                            __syncwarp();
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const int row8 = j * 8 + (lane >> 2);
                                uint4 v;
                                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                             : "r"(room + row8 * 64 + (((lane & 3) ^ ((row8 >> 1) & 3)) << 4)));
                                if (to[j] >= 0) *reinterpret_cast<uint4 *>(base + to[j] * kLatent + q * 128) = v;
                            }
                            __syncwarp();  // read before the next is written
                        }
                    }
                } else {
                    // a thread stores its channel of each row, 128 bytes of a row together in a warp
                    uint8_t *base = static_cast<uint8_t *>(p.o) + (warp * 32 + lane) * 4;
#pragma unroll 1
                    for (int r0 = 0; r0 < (int)q_rows; r0 += 16) {
                        float o[64], f[16];
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_ld16f(tb + lane_base + kTmemO + q * pl.n + r0, o + 16 * q);
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = b.factor[r0 + i];
                        wait_ld<64>(o);
                        if (nt == 0) {
#pragma unroll
                            for (int i = 0; i < 64; ++i) o[i] = 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int64_t row_at = b.row_at[r0 + i];
                            uint8_t *at = base + row_at * (kLatent * 4);
#pragma unroll
                            for (int q = 0; q < 4; ++q) store_if(row_at >= 0, at + q * 512, o[16 * q + i] * f[i]);
                        }
                    }
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b.i_empty + k % kSlots);
                if (nt > 0) mbar_arrive(&b.o_free);
            }
            items += nt > 0;
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kScoreWarp) tmem_dealloc(tb, 512);
    // After a failure every row of this CTA's items becomes NaN.
    if (*abort_flag) {
        Walk w;
        w.start(a, way, whole, L0, L1, S, pad, start_seq, start_begin, start_unit);
        for (;;) {
            const Item it = w.next(a, piece, g, threadIdx.x == 0);
            if (!it.found) break;
            if (it.part >= 0) {
                for (int i = threadIdx.x; i < part_floats(pl); i += kThreads) p.ws[it.part + i] = kNaN;
                continue;
            }
            for (int i = threadIdx.x; i < (int)q_rows * kLatent; i += kThreads) {
                const int r = i / kLatent, ch = i - r * kLatent, tok = r / pl.hp, head = it.head0 + r - tok * pl.hp;
                if (tok >= it.tokens || head >= p.H) continue;
                const int64_t out = (int64_t)(it.t0 + tok) * p.H + head;
                st_out(p.o, out * kLatent + ch, kNaN, p.o_bf16);
                if (ch == 0 && p.lse) p.lse[out] = kNaN;
            }
        }
        if (pl.cut && threadIdx.x == 0) last_words(w);
        if (threadIdx.x == 0) atomicAdd(&g_attn_latent_timeouts, 1);
    }
}

// Joins the tiles that more than one piece took, in the order of the pieces.  blockIdx.x is a unit's tile, or
// with more units than pieces a CTA of the first launch, which looks after the tile that begins in its
// piece and goes on behind it, if there is one.  A warp has four rows and 128 channels, or with
// `shares` > 1 a share of their pieces.
constexpr int kMaxShares = 4;
__global__ void __launch_bounds__(128 * kMaxShares) attn_latent_join_kernel(const __grid_constant__ Args a, int shares) {
    extern __shared__ float4 s_acc[];  // [shares - 1 of 4 warps][128], then their m and l
    const AttnLatentParams &p = a.p;
    const Plan &pl = a.plan;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 *words = join_words(a);
    const int4 of = __ldcg(words + words_of(pl)), word = __ldcg(words + blockIdx.x);
    const int G = of.y, which = blockIdx.x / G, g = blockIdx.x - which * G;
    const JoinWord t = *reinterpret_cast<const JoinWord *>(&word);
    const int share = warp >> 2, q = warp & 3, k0 = t.first, k1 = t.last;
    const int r = 4 * blockIdx.y;  // the first of the rows
    if (which >= of.x || k0 >= k1) return;
    int64_t out[4];  // their places, or -1
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int tok = (r + e) / pl.hp, head = (t.place & 0xFFFF) + r + e - tok * pl.hp;
        out[e] = tok < t.place >> 16 && head < p.H ? (int64_t)(t.t0 + tok) * p.H + head : -1;
    }
    if (max(max(out[0], out[1]), max(out[2], out[3])) < 0) return;
    float m[4], l[4], acc[4][4];  // of the rows; of channels lane + 32 * i
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        m[e] = -INFINITY;
        l[e] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][e] = 0.f;
    }
    const int each = (k1 - k0 + shares) / shares, from = k0 + share * each, to = min(from + each, k1 + 1);
    // (the tile is in slot 1 of the piece that it begins in, else in slot 0)
    const int64_t floats = part_floats(pl), step = 2 * G * floats;
    const float *ws = p.ws + (from * G + g) * 2 * floats + (share == 0 ? floats : 0);
    const int at = pl.n * kLatent + r;
    struct Four {
        float4 m, l, x[4];
    } now, next;
    auto load = [&](Four &f, const float *ws) {
        const float4 *x = reinterpret_cast<const float4 *>(ws + ((int64_t)(q * pl.n + r) / 4 * 128 + lane) * 4);
        f.m = __ldcg(reinterpret_cast<const float4 *>(ws + at));
        f.l = __ldcg(reinterpret_cast<const float4 *>(ws + at + pl.n));
#pragma unroll
        for (int i = 0; i < 4; ++i) f.x[i] = __ldcg(x + 32 * i);
    };
    if (from < to) load(next, ws);
    for (int k = from; k < to; ++k) {  // every lane forms the factors itself: the next part is on its way meanwhile
        now = next;
        if (k == k0) ws -= floats;
        ws += step;
        if (k + 1 < to) load(next, ws);
        const float mk[4] = {now.m.x, now.m.y, now.m.z, now.m.w}, lk[4] = {now.l.x, now.l.y, now.l.z, now.l.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float most = fmaxf(m[e], mk[e]), own = most == -INFINITY ? 1.f : ex2(m[e] - most);
            const float f = most == -INFINITY ? 1.f : ex2(mk[e] - most);
            m[e] = most;
            l[e] = fmaf(lk[e], f, l[e] * own);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = e == 0 ? now.x[i].x : e == 1 ? now.x[i].y : e == 2 ? now.x[i].z : now.x[i].w;
                acc[i][e] = fmaf(x, f, acc[i][e] * own);
            }
        }
    }
    if (shares > 1) {  // the first four warps add the others' sums to theirs
        float4 *s_m = s_acc + (shares - 1) * 4 * 128, *s_l = s_m + (shares - 1) * 4;
        if (share > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) s_acc[(warp - 4) * 128 + lane + 32 * i] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            if (lane == 0) s_m[warp - 4] = make_float4(m[0], m[1], m[2], m[3]), s_l[warp - 4] = make_float4(l[0], l[1], l[2], l[3]);
        }
        __syncthreads();
        if (share > 0) return;
        for (int w = q; w < (shares - 1) * 4; w += 4) {
            const float4 x = s_m[w], y = s_l[w];
            const float mw[4] = {x.x, x.y, x.z, x.w}, lw[4] = {y.x, y.y, y.z, y.w};
            float f[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float most = fmaxf(m[e], mw[e]), own = most == -INFINITY ? 1.f : ex2(m[e] - most);
                f[e] = most == -INFINITY ? 1.f : ex2(mw[e] - most);
                m[e] = most;
                l[e] = fmaf(lw[e], f[e], l[e] * own);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][e] *= own;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = s_acc[w * 128 + lane + 32 * i];
                acc[i][0] = fmaf(v.x, f[0], acc[i][0]);
                acc[i][1] = fmaf(v.y, f[1], acc[i][1]);
                acc[i][2] = fmaf(v.z, f[2], acc[i][2]);
                acc[i][3] = fmaf(v.w, f[3], acc[i][3]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (out[e] < 0) continue;
        const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
#pragma unroll
        for (int i = 0; i < 4; ++i) st_out(p.o, out[e] * kLatent + q * 128 + lane + 32 * i, acc[i][e] * inv, p.o_bf16);
        if (q == 0 && lane == 0 && p.lse) p.lse[out[e]] = l[e] == 0.f ? -INFINITY : (log2f(l[e]) + m[e]) * kLn2;
    }
}

// ---------------------------------------------------------------------------
// host

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// The tiles that read a sequence together, of sequences of `tiles`: as many as leave at most kIdle more of the CTAs
// without a tile than the best does.  More of them read the cache fewer times: 16 sequences of 10000 tokens with
// 4 rows, 64 heads (4 tiles), by 1, 2 and 4: 125, 108 and 104 us.  But what does not divide the tiles idles: with 5
// rows by 1, 2, 4 and 5: 138, 151, 185 and 126 us.
int share_of(int64_t tiles) {
    const int sms = sm_count(), most = std::min(kMaxShare, sms);
    auto cost = [&](int G) { return (double)((tiles + G - 1) / G) / (sms / G); };
    double least = cost(1);
    for (int G = 2; G <= most; ++G) least = std::min(least, cost(G));
    int G = most;
    while (cost(G) > (1. + kIdle) * least) --G;
    return G;
}

// How a call is split.  Tiles: all heads of as many tokens as 64 rows hold, or with more than 64 heads
// equal parts of one token's.  (Heads filled up to eight, as a tile's blocks need, wasted rows: 13 sequences of 81 rows, 2
// heads 696 and now 193 us; 64 of 5 rows, 12 heads 60 and 50.)
Plan plan_of(int64_t N, int64_t tokens, int H, int64_t max_tokens) {
    Plan pl;
    memset(&pl, 0, sizeof(pl));
    const int64_t avg = (tokens + N - 1) / N;  // rows of a sequence
    pl.parts = (H + kTileRows - 1) / kTileRows;
    pl.hp = (H + pl.parts - 1) / pl.parts;
    pl.tk = (int)std::max<int64_t>(1, std::min<int64_t>(kTileRows / pl.hp, avg));
    pl.n = (int)round_up(pl.hp * pl.tk, 16);
    pl.q_rows = (int)round_up(pl.hp * pl.tk, 8);
    const int64_t tiles = (avg + pl.tk - 1) / pl.tk * pl.parts;
    // A token's tiles are shared in either way; a sequence's too where all have about as many rows.
    pl.G[0] = share_of(pl.parts);
    pl.G[1] = share_of(tiles);
    int64_t most_units[2], sms[2];
    for (int w = 0; w < 2; ++w) {
        sms[w] = std::max(sm_count() / pl.G[w], 1);
        pl.units_one[w] = (pl.parts + pl.G[w] - 1) / pl.G[w];
        // (a sequence of nq rows has at most nq / (rows of a unit) + 1 units)
        most_units[w] = tokens == N ? N * units_of(pl, w, 1) : units_of(pl, w, (int)tokens) + N;
    }
    const int64_t per = (max_tokens + kStep - 1) / kStep;
    // Units are cut where that balances more than it costs (the sums' way through L2 and the second launch).  The lengths
    // are not known here, only the table's width: where it says enough, the second launch falls away.  Cut and whole,
    // 32 heads: 16 sequences of at most 256, 512, 1024 tokens 14.3 and 11.7, 15.9 and 15.8, 17.8 and 24.0 us; 76 of 1024,
    // 2048 tokens 30.8 and 27.3, 44.4 and 45.4; 128 of 1024, 2048, 4096 tokens 37.7 and 32.6, 59.2 and 54.3, 108 and 96,
    // but of 100 to 4096 tokens 68.0 and 82.8.
    pl.cut = !(most_units[0] <= sms[0] && (per <= 4 || per * sms[0] <= 44 * most_units[0]));
    if (!pl.cut) pl.G[1] = pl.G[0], pl.units_one[1] = pl.units_one[0], most_units[1] = most_units[0];
    for (int w = 0; w < 2; ++w) {
        pl.pieces[w] = (int)(pl.cut ? std::max<int64_t>(1, std::min(sms[w], most_units[w] * per)) : most_units[w]);
        pl.ctas = std::max(pl.ctas, pl.pieces[w] * pl.G[w]);
        pl.most_places = std::max(pl.most_places, most_units[w] * pl.G[w]);
    }
    pl.by_unit = pl.most_places < pl.ctas;
    // Up to 48 rows leave TMEM for a third unit of the queries, and so the ring a place more, which longer calls gain from:
    // with two and three units in TMEM 8 sequences of 60000 tokens, 96 heads 140 and 134 us, 128 of 1000, 32 heads 35.1 and
    // 33.9, but 32 of 300 12.6 and 13.1, 64 of 5 8.8 and 9.4 (three units take longer to come).
    pl.q_units = pl.n <= 48 && pl.most_places * per >= (int64_t)8 * pl.ctas ? 1 : 2;
    const int64_t q = (int64_t)pl.q_rows * (2 * pl.q_units + 1) * 128;
    const int64_t ps = std::max<int64_t>(pl.n * 128, kSoftWarps * 1024);  // (the output is turned there, too)
    const int64_t room = kMaxSmem - 1024 - (int64_t)round_up(sizeof(Bars), 128) - round_up(q, 1024) - round_up(ps, 1024);
    pl.units = (int)std::min<int64_t>(kMaxUnits, (room - kShared * kSharedBytes) / kUnitBytes);
    pl.at_p = (uint32_t)round_up(q, 1024);
    pl.at_units = pl.at_p + (uint32_t)round_up(ps, 1024);
    pl.at_shared = pl.at_units + pl.units * kUnitBytes;
    pl.at_bars = pl.at_shared + kShared * kSharedBytes;
    return pl;
}

size_t plan_bytes(const Plan &pl) {
    return pl.cut ? (size_t)pl.ctas * 2 * part_floats(pl) * sizeof(float) + (words_of(pl) + 1) * sizeof(JoinWord) : 0;
}

bool encode_tensors(const AttnLatentParams &p, const Plan &pl, CUtensorMap *mq, CUtensorMap *mc, CUtensorMap *mr) {
    chunk::EncodeTiledFn enc = reinterpret_cast<chunk::EncodeTiledFn>(tensor_map_encoder());
    if (!enc) {
        set_error("attn_latent: cuTensorMapEncodeTiled is not available from the driver");
        return false;
    }
    const cuuint32_t es[3] = {1, 1, 1};
    const cuuint64_t qd[3] = {(cuuint64_t)kRow, (cuuint64_t)p.H, (cuuint64_t)p.tokens};
    const cuuint64_t qs[2] = {(cuuint64_t)kRow * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t qb[3] = {64, (cuuint32_t)pl.hp, (cuuint32_t)pl.tk};
    CUresult r = enc(mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(p.q), qd, qs, qb, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    // The cache as [9 blocks of 64 channels][rows][64]: a copy brings two blocks of a step's rows (mc), or one of
    // a small page's (mr), each block's rows together as the products take them.
    const cuuint64_t cd[3] = {64, (cuuint64_t)p.c.n_pages * p.c.P, kRow / 64};
    const cuuint64_t cs[2] = {(cuuint64_t)kRow * 2, 128};
    for (int blocks = 1; blocks <= 2 && r == CUDA_SUCCESS; ++blocks) {
        const cuuint32_t cb[3] = {64, (cuuint32_t)std::min(p.c.P, kStep), (cuuint32_t)blocks};
        r = enc(blocks == 1 ? mr : mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.c.rows, cd, cs, cb, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    }
    if (r != CUDA_SUCCESS) set_error("attn_latent: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return r == CUDA_SUCCESS;
}

}  // namespace

int take_attn_latent_timeouts(cudaStream_t st) {
    int n = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&n, g_attn_latent_timeouts, sizeof(int), 0, cudaMemcpyDeviceToHost, st) !=
            cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_attn_latent_timeouts, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) !=
            cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        set_error("attn_latent: cannot read the timeout counter: %s", cudaGetErrorString(cudaGetLastError()));
        return -1;
    }
    return n;
}

size_t attn_latent_workspace_bytes(int64_t N, int64_t tokens, int H, int64_t max_tokens) {
    return plan_bytes(plan_of(N, tokens, H, max_tokens));
}

kda_status launch_attn_latent(const AttnLatentParams &p, cudaStream_t st) {
    if (p.tokens == 0 || p.c.N == 0) return KDA_OK;
    Args a;
    memset(&a, 0, sizeof(a));
    a.p = p;
    a.plan = plan_of(p.c.N, p.tokens, p.H, (int64_t)p.c.max_blocks * p.c.P);
    const Plan &pl = a.plan;
    CUtensorMap mq, mc, mr;
    if (!encode_tensors(p, pl, &mq, &mc, &mr)) return KDA_ERR_CUDA;
    static DeviceOnce configured;
    const int dev = current_device();
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(attn_latent_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess ||
            cudaFuncSetAttribute(attn_latent_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) {
            set_error("attn_latent: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];  // either launch starts while the one before ends, and waits for it before it reads
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(pl.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, pl.q_units == 1 ? attn_latent_kernel<1> : attn_latent_kernel<2>, mq, mc, mr, a);
    note_launch();
    if (e != cudaSuccess) {
        set_error("attn_latent_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    kda_status s = check_launch("attn_latent_kernel");
    if (!pl.cut || s != KDA_OK) return s;
    // with many pieces a unit more warps share them
    const int shares = pl.ctas >= 16 * pl.most_places ? kMaxShares : 1;
    cfg.gridDim = dim3((unsigned)words_of(pl), (pl.hp * pl.tk + 3) / 4);
    cfg.blockDim = dim3(128 * shares);
    cfg.dynamicSmemBytes = (shares - 1) * 4 * (128 + 2) * sizeof(float4);
    e = cudaLaunchKernelEx(&cfg, attn_latent_join_kernel, a, shares);
    note_launch();
    if (e != cudaSuccess) {
        set_error("attn_latent_join_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return check_launch("attn_latent_join_kernel");
}

}  // namespace kda
