// kda_attn_prompt.cu -- causal attention over whole prompts, packed sequences of different
// lengths, grouped heads; on the tensor cores.
//
//   o_i = sum_{j < seen_i} softmax_j(scale * q_i . k_j) v_j,   seen_i = i + 1 + (keys - queries)
//
// Flash form: key blocks of 128 tokens pass by, and each row keeps a reference m, the sum l
// of 2^(s - m) and the weighted sum O of the values (s the scores in units of log2).  m is the
// row's maximum when it was last set, at first that of its first block of 128 keys (of its part's,
// where the keys are divided); it is set anew (and l, O brought to it) only when a score exceeds it
// by more than kSlack.  Weights, l and O are all
// floating, so which m is used costs no precision, and O is hardly ever touched.
//
// A CTA takes two query tiles of 128 rows: two heads of one key/value head where the group
// is even (both read the same keys), else 256 consecutive rows of one head.
//   warps 0-3, 4-7  softmax of tile 0 / 1, a thread per row: scores from TMEM, weights
//                   rounded to bf16 back into TMEM over the scores, in two halves, so that
//                   the product with the first half's values runs beside the second's weights
//   warps 8, 9      issue the products of tile 0 / 1: S_t = Q_t K^T (both operands in shared
//                   memory) and O_t += P_t V (P from TMEM).  They take turns, a tile's O and
//                   next S together, so that one tile's softmax runs beside the other's
//                   products; a warp has done its waiting (100 to 200 cycles a barrier) when
//                   its turn comes
//   warp 10         TMA: the query tiles, and rings of key and value blocks
//   warp 11         finds the next work items
// CTAs are persistent, one per SM; work items (a run of query rows of a sequence, and a head
// or a pair; with few of them also a part of their keys) are taken longest first, in rounds of
// alternating direction.  Loads, scores and
// rings go on across items, so that an item's beginning runs beside the last one's end.
// TMEM: S_0, S_1 (P over them), O_0, O_1, 128 columns each; with 64 channels O takes 64, and P has
// columns of its own, so that a block's scores are formed while the softmax works on the last ones
// and the product warps need no turns (8192 tokens 275 -> 254 us).
//
// Weights are rounded to bf16 because the product takes one type and the values are bf16;
// l sums the unrounded weights in fp32.
//
// 8192 tokens with 32 heads over 8, channels 64/64, 128/128, 192/128: 254, 316, 400 us, 1082, 1740 and
// 1718 TFLOP/s in runs of a few passes; in long runs the power limit lowers the clock (2400 passes of
// 128/128: 339 us at 1740 MHz).  With 128 and more channels the tensor pipe is busy for 70 to 75 % of the
// cycles and a tile's chain of scores, softmax and product is the bound; with 64, where a weight
// comes for 256 operations instead of 512 or 640, that chain too: the tensor pipe is busy for 42 %
// of the cycles, the special functions' for 42 %, the issue slots for 44 % (4096 tokens).  8 packed
// prompts of [100, 4096] tokens, 32 heads of 192/128: 125 to 132 us (tensor pipe 56 %), where each
// item's beginning and end (about 4 us of queries, first scores and output) count.  100 tokens: 6.8 us.
//
// What is masked never reaches a result: masked scores are replaced, not added to; value
// rows behind the sequence's end are zeroed in shared memory (a zero weight would turn an
// infinity there into NaN); where a row comes out NaN and a value of a later token of its own
// blocks caused it, the channels concerned are computed alone (rescue_row), when the
// CTA's items are through: such a row may see any number of keys, and no bounded wait may run meanwhile.
#include <cuda.h>
#include <string.h>

#include <algorithm>

#include "kda_attn.cuh"
#include "kda_chunk_common.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kTile = 128;             // query rows of a tile, and keys of a block
constexpr int kMmaWarp = 8, kTmaWarp = 10, kItemWarp = 11;
constexpr int kThreads = 384;
constexpr int kFewRegs = 120, kManyRegs = 192;  // a thread's registers in warps 8-11 and 0-7
constexpr int kLaunchRegs = 168;                // and at launch, which must cover them
static_assert(kFewRegs * 128 + kManyRegs * 256 <= kLaunchRegs * kThreads, "a larger share would be waited for without end");
constexpr int kItemReaders = 11;       // warps that follow the work items
constexpr float kSlack = 40.f;         // log2: how far a score may exceed the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ int g_attn_prompt_timeouts = 0;

template <int D, int DV>
struct Cfg {
    // A block's values come whole, or with 192 channels, where shared memory holds one block of
    // them, in two halves, each free for its successor when both tiles' products have read it.
    static constexpr int NV = D == 192 ? 2 : 1, VROWS = kTile / NV;
    static constexpr uint32_t QB = kTile * D * 2, KB = kTile * D * 2, VB = VROWS * DV * 2;
    static constexpr int KST = D == 64 ? 4 : 2, VST = D == 64 ? 4 : 2;
    static constexpr uint32_t Q = 0, K = 2 * QB, V = K + KST * KB, BARS = V + VST * VB;
    static constexpr int NBAR = 4 + 2 * KST + 2 * VST + 1 + 2 + 4 + 2 + 2 + 4 + 4;
    static constexpr uint32_t SMEM = BARS + NBAR * 8 + 96 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    // TMEM columns of tile 0's scores, output and weights.  Where the output is narrow the weights have
    // columns of their own: a block's scores are then formed while the softmax works on the last
    // ones (254 against 275 us for 8192 tokens, 32/8 heads of 64); else they lie over the scores.
    static constexpr bool AHEAD = 2 * (kTile + DV + kTile / 2) <= 512;
    static constexpr uint32_t T_S = 0, T_O = 2 * kTile, T_P = AHEAD ? T_O + 2 * DV : T_S;
    static constexpr uint32_t P_STEP = AHEAD ? kTile / 2 : kTile;  // from tile 0's weights to tile 1's
};

struct Args {
    PromptParams p;
    int pair_heads;  // 1: two heads of a group share their rows; 0: 256 rows of one head
    int n_heads;     // work items per unit: head pairs, or heads
    int items;       // work items at most
    int parts;       // work items of a unit and head, each with its share of the key blocks
};

// Query and key rows of a sequence.
struct Seq {
    int q0, nq, k0, nk;
};
struct Item {
    Seq s;
    int found, row0, head;  // head: number of the pair, or of the head
    int lo, hi, place;      // in the form with parts: its key blocks [lo, hi), and where its sums go
};

// What a part leaves in the workspace: the 2 x 128 rows' O, their m and their l.
template <int DV>
constexpr int kPartFloats = 2 * kTile * (DV + 2);

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}
// A TMA load with a priority in L2: queries are read once and leave first, keys and values are
// read again by other work items.
__device__ __forceinline__ void tma_load_hint(uint32_t dst, const void *tmap, uint64_t *bar, int x, int y, int z, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, "
        "%4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t leave_first() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t leave_last() {
    uint64_t p;
    asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Waits for the loads issued so far; naming the registers keeps their uses behind the wait.
__device__ __forceinline__ void wait_ld64(float *r) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 64; i += 16)
        asm volatile("" : "+f"(r[i]), "+f"(r[i + 1]), "+f"(r[i + 2]), "+f"(r[i + 3]), "+f"(r[i + 4]), "+f"(r[i + 5]),
                     "+f"(r[i + 6]), "+f"(r[i + 7]), "+f"(r[i + 8]), "+f"(r[i + 9]), "+f"(r[i + 10]), "+f"(r[i + 11]),
                     "+f"(r[i + 12]), "+f"(r[i + 13]), "+f"(r[i + 14]), "+f"(r[i + 15]));
}
// 32 columns from two runs of 16 registers.
__device__ __forceinline__ void tmem_st16x2(uint32_t taddr, const float *r, const float *q) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
        "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(q[0]), "f"(q[1]), "f"(q[2]),
        "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]), "f"(q[8]), "f"(q[9]), "f"(q[10]), "f"(q[11]), "f"(q[12]),
        "f"(q[13]), "f"(q[14]), "f"(q[15])
        : "memory");
}

// One lane of a converged warp, always the same one.  The compiler knows that a branch on it
// has a single active thread, so that the tensor instructions in it are issued back to back;
// under `lane == 0` each cost about 130 cycles instead of 64 (M = N = 128, K = 16).
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// 4 x 4 matrix of 16-byte pieces over four neighbouring lanes, transposed: lane i's piece q
// becomes lane q's piece i.
__device__ __forceinline__ void transpose_quad(uint32_t (&w)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q & m) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t give = up ? w[4 * q + e] : w[4 * (q | m) + e];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, give, m);
                if (up)
                    w[4 * q + e] = got;
                else
                    w[4 * (q | m) + e] = got;
            }
        }
    }
}

// The weights stored so far are in TMEM: tells the products' warp (one arrival per warp).
__device__ __forceinline__ void hand_over(uint64_t *bar) {
    tmem_wait_st();
    fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A barrier of two warps that also says whether any of their threads has `x`.
__device__ __forceinline__ bool pair_any(int id, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(id)
        : "memory");
    return r != 0;
}

// The turn of the product warps: barrier 1 gives it to tile 0's, barrier 2 to tile 1's.
__device__ __forceinline__ void turn_wait(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void turn_pass(int id) { asm volatile("barrier.cta.arrive %0, 64;" ::"r"(id) : "memory"); }

// A 128-byte-swizzled operand's descriptor from its low word (address / 16 and leading offset);
// the row groups are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sequence n, clamped to the tensors.
__device__ __forceinline__ Seq seq_of(const PromptParams &p, int n) {
    auto range = [&p](const int32_t *cu, int n, int64_t T, int &at, int &len) {
        if (!cu) {  // equal lengths
            len = (int)(T / p.N);
            at = n * len;
            return;
        }
        int64_t a = __ldg(cu + n), b = __ldg(cu + n + 1);
        a = max((int64_t)0, min(a, T));
        b = max(a, min(b, T));
        at = (int)a;
        len = (int)(b - a);
    };
    Seq s;
    range(p.cu_q, n, p.Tq, s.q0, s.nq);
    range(p.cu_k, n, p.Tk, s.k0, s.nk);
    return s;
}

// Work units, runs of 2^shift query rows of one sequence, longest first: one warp's search, asked
// for ever higher ranks.  A unit's level is the number of keys its first row sees, above the
// smallest of any first unit and in units of 2^shift, so that a sequence has units on as many levels
// as it has units, one each.  The warp holds 128 sequences, and takes the next 128 when those
// are through (the order then holds within them).
struct UnitSearch {
    int next = 0;               // first sequence not taken yet
    int before = 0, total = 0;  // units of the sequences before those held, and of those
    int top = 0;                // no unit asked for from now on lies above this level
    int all[4], base[4];        // a lane's sequences: their units, and the first one's level

    __device__ int above(int level) const {  // held units at or above a level
        int c = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) c += all[e] - min(max(level - base[e], 0), all[e]);
        return __reduce_add_sync(0xffffffffu, c);
    }
    __device__ void take(const PromptParams &p, int shift) {
        const int lane = threadIdx.x & 31;
        int more[4], least = INT_MAX, units = 0, levels = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int n = next + e * 32 + lane;
            all[e] = more[e] = 0;
            if (n >= p.N) continue;
            const Seq s = seq_of(p, n);
            all[e] = (int)(((int64_t)s.nq + (1 << shift) - 1) >> shift);
            more[e] = s.nk - s.nq;
            if (all[e]) least = min(least, more[e]);
        }
        least = __reduce_min_sync(0xffffffffu, least);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            base[e] = all[e] ? (int)(((uint32_t)more[e] - (uint32_t)least) >> shift) : 0;
            units += all[e];
            levels = max(levels, base[e] + all[e]);
        }
        before += total;
        total = __reduce_add_sync(0xffffffffu, units);
        top = __reduce_max_sync(0xffffffffu, levels) - 1;
        next += 128;
    }
    // The rank-th unit: its sequence and first row; false if there are fewer.
    __device__ bool find(const PromptParams &p, int shift, int rank, int &seq, int &row0) {
        if (!p.cu_q) {  // equal lengths: round by round
            const int nq = (int)(p.Tq / p.N), u = ((nq + (1 << shift) - 1) >> shift) - 1 - rank / p.N;
            seq = rank % p.N;
            row0 = u << shift;
            return u >= 0;
        }
        if (p.N == 1) {
            if (!next) all[0] = (seq_of(p, 0).nq + (1 << shift) - 1) >> shift, next = 1;
            seq = 0;
            row0 = (all[0] - 1 - rank) << shift;
            return row0 >= 0;
        }
        while (rank >= before + total) {
            if (next >= p.N) return false;
            take(p, shift);
        }
        rank -= before;
        int lo = 0;  // the highest level with more than `rank` units from it on
        while (lo < top) {
            const int m = (lo + top + 1) >> 1;
            if (above(m) > rank)
                lo = m;
            else
                top = m - 1;
        }
        int left = rank - above(lo + 1);  // in the order of the sequences
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int u = lo - base[e];
            const bool has = u >= 0 && u < all[e];
            const uint32_t who = __ballot_sync(0xffffffffu, has);
            const uint32_t it = __ballot_sync(0xffffffffu, has && __popc(who & ((1u << lane) - 1)) == left);
            if (it) {
                const int src = __ffs(it) - 1;
                seq = next - 128 + e * 32 + src;
                row0 = __shfl_sync(0xffffffffu, u, src) << shift;
                return true;
            }
            left -= __popc(who);
        }
        return false;
    }
};

// First row of an item's tile t.
__device__ __forceinline__ int first_row(const Args &a, const Item &it, int t) {
    return a.pair_heads ? it.row0 : it.row0 + t * kTile;
}
// Key blocks of an item that its tile t sees.
template <bool SPLIT>
__device__ __forceinline__ int blocks_of(const Args &a, const Item &it, const Seq &s, int t) {
    const int r = first_row(a, it, t), last = min(r + kTile, s.nq) - 1;
    if (r >= s.nq) return 0;
    const int seen = max(0, min(s.nk, last + 1 + (s.nk - s.nq)));
    const int n = (seen + kTile - 1) / kTile;
    return SPLIT ? max(0, min(n, it.hi) - it.lo) : n;
}
// This CTA's k-th work item; one warp.
template <bool SPLIT>
__device__ __forceinline__ Item item_of(const Args &a, UnitSearch &units, int k) {
    const int64_t i = (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    const int u = SPLIT ? (int)i / a.parts : (int)i, part = SPLIT ? (int)i - u * a.parts : 0;
    Item it = {{0, 0, 0, 0}, 0, 0, u % a.n_heads, 0, INT_MAX, (int)i};
    int seq = 0;
    if (i < a.items) it.found = units.find(a.p, a.pair_heads ? 7 : 8, u / a.n_heads, seq, it.row0);
    if (it.found) it.s = seq_of(a.p, seq);
    if (SPLIT && it.found) {
        const int nb = max(blocks_of<SPLIT>(a, it, it.s, 0), blocks_of<SPLIT>(a, it, it.s, 1));
        it.lo = (int)((int64_t)nb * part / a.parts);
        it.hi = (int)((int64_t)nb * (part + 1) / a.parts);
    }
    return it;
}

// Weights 2^(c y - m) of 32 scores y, left as bf16 pairs in the words y[0, 16); their sum is
// added to s (two pairs of halves).
__device__ __forceinline__ void weights32(float *y, float c, float m, float2 (&s)[2]) {
    const float mm = m == -INFINITY ? 0.f : m;  // a row that has seen nothing: every score is -inf
    const float2 c2 = make_float2(c, c), m2 = make_float2(-mm, -mm);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float2 e = fma2(make_float2(y[2 * i], y[2 * i + 1]), c2, m2);
        e.x = ex2(e.x);
        e.y = ex2(e.y);
        s[i & 1] = add2(s[i & 1], e);
        y[i] = __uint_as_float(pack_bf16x2(e.x, e.y));
    }
}

// A row's channels that a masked value spoiled, computed alone by one warp over the keys
// [from, seen) that the row sees; its tile went through the keys up to `end`.  c: the scale in
// units of log2; part: a part's O of this row, whose reference is part_m, or null.  A row that is
// finite, or whose masked values are, is left as it is.  The pass goes backwards and ends when
// every channel concerned is NaN by what the row sees, as behind the valid part of a padded sequence.
template <int D, int DV>
__device__ __forceinline__ void rescue_row(const PromptParams &p, const Seq &s, int row, int head, int from, int seen, int end,
                                        float c, float *part, float part_m) {
    constexpr int C = DV / 32;  // channels of a lane
    constexpr uint32_t kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31, kvh = head / (p.Hq / p.Hk), d0 = lane * C;
    const int64_t out = ((int64_t)(s.q0 + row) * p.Hq + head) * DV + d0;
    const __nv_bfloat16 *v0 = p.v + (int64_t)s.k0 * p.v_stride + (int64_t)kvh * DV + d0;
    uint32_t odd = 0, bad = 0;  // bits: outputs that are not finite, and among them masked values that are not
#pragma unroll
    for (int e = 0; e < C; ++e) {
        const float x = part ? part[d0 + e]
                             : p.o_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.o)[out + e])
                                        : static_cast<const float *>(p.o)[out + e];
        odd |= (uint32_t)!isfinite(x) << e;
    }
    if (!__any_sync(kAll, odd != 0)) return;
    for (int j = max(seen, from); j < end; ++j)
#pragma unroll
        for (int e = 0; e < C; ++e) bad |= (uint32_t)!isfinite(__bfloat162float(v0[j * p.v_stride + e])) << e;
    bad &= odd;
    if (!__any_sync(kAll, bad != 0)) return;
    const uint4 *q = reinterpret_cast<const uint4 *>(p.q + (int64_t)(s.q0 + row) * p.q_stride + (int64_t)head * D);
    const __nv_bfloat16 *k0 = p.k + (int64_t)s.k0 * p.k_stride + (int64_t)kvh * D;
    float acc[C] = {}, m = -INFINITY, l = 0.f;
    for (int j1 = seen; j1 > from; j1 -= 32) {
        const int j0 = max(from, j1 - 32), n = j1 - j0;
        float score = -INFINITY;  // of this lane's key
        if (lane < n) {
            const uint4 *k = reinterpret_cast<const uint4 *>(k0 + (j0 + lane) * p.k_stride);
            float dot = 0.f;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                float a[8], b[8];
                Vec16<__nv_bfloat16>::load(__ldg(q + i), a);
                Vec16<__nv_bfloat16>::load(__ldg(k + i), b);
#pragma unroll
                for (int e = 0; e < 8; ++e) dot = fmaf(a[e], b[e], dot);
            }
            score = dot * c;
        }
        float most = score;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, o));
        most = fmaxf(most, m);
        const float f = most == -INFINITY ? 1.f : ex2(m - most), w = ex2(score - (most == -INFINITY ? 0.f : most));
        m = most;
        float sum = w;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
        l = fmaf(l, f, sum);
#pragma unroll
        for (int e = 0; e < C; ++e) acc[e] *= f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const float wi = __shfl_sync(kAll, w, i);
#pragma unroll
            for (int e = 0; e < C; ++e) acc[e] = fmaf(wi, __bfloat162float(v0[(j0 + i) * p.v_stride + e]), acc[e]);
        }
        bool open = false;
#pragma unroll
        for (int e = 0; e < C; ++e) open |= (bad >> e & 1) && !isnan(acc[e]);
        if (!__any_sync(kAll, open)) break;
    }
    const float f = part ? (m == -INFINITY ? 0.f : ex2(m - part_m)) : l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < C; ++e) {
        if (!(bad >> e & 1)) continue;
        if (part)
            part[d0 + e] = acc[e] * f;
        else
            st_out(p.o, out + e, acc[e] * f, p.o_bf16);
    }
}

// The same for the rows of all of a softmax warp's items, which it has written.
template <int D, int DV, bool SPLIT>
__device__ __forceinline__ void rescue_rows(const Args &a) {
    const PromptParams &p = a.p;
    const int warp = threadIdx.x >> 5, t = warp >> 2;
    UnitSearch units;
    for (int k = 0;; ++k) {
        const Item it = item_of<SPLIT>(a, units, k);
        if (!it.found) break;
        const Seq s = it.s;
        const int row0 = first_row(a, it, t), head = a.pair_heads ? 2 * it.head + t : it.head;
        const int from = SPLIT ? it.lo * kTile : 0, end = min(s.nk, from + blocks_of<SPLIT>(a, it, s, t) * kTile);
        float *part = SPLIT ? p.ws + (int64_t)it.place * kPartFloats<DV> : nullptr;
        for (int r = (warp & 3) * 32; r < (warp & 3) * 32 + 32 && row0 + r < s.nq; ++r) {
            const int seen = max(0, min(end, row0 + r + 1 + s.nk - s.nq));
            if (SPLIT && seen <= from) continue;  // the part's sums of this row are not read
            rescue_row<D, DV>(p, s, row0 + r, head, from, seen, end, p.scale * kLog2e,
                              SPLIT ? part + (t * kTile + r) * DV : nullptr,
                              SPLIT ? part[2 * kTile * DV + t * kTile + r] : 0.f);
        }
    }
}

template <int D, int DV, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args a) {
    using L = Cfg<D, DV>;
    const PromptParams &p = a.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm), sb16 = sb >> 4;
    uint64_t *q_full = reinterpret_cast<uint64_t *>(sm + L::BARS), *q_empty = q_full + 2;  // [2] each
    uint64_t *k_full = q_empty + 2, *k_empty = k_full + L::KST;
    uint64_t *v_full = k_empty + L::KST, *v_empty = v_full + L::VST;
    uint64_t *v_raw = v_empty + L::VST;                             // a last value block, before its tail is zeroed
    uint64_t *s_full = v_raw + 1, *p_ready = s_full + 2;            // p_ready[tile * 2 + half]
    uint64_t *o_full = p_ready + 4, *drain = o_full + 2;
    uint64_t *i_full = drain + 2, *i_empty = i_full + 2;            // the work items' two slots
    uint64_t *s_free = i_empty + 2, *p_free = s_free + 2;           // scores read; weights multiplied (AHEAD)
    Item *slots = reinterpret_cast<Item *>(p_free + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(slots + 2);
    volatile int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);  // a bounded wait gave up
    volatile int *spoiled = abort_flag + 1;  // a row came out NaN
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (SPLIT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(q_full + i, 1);
            mbar_init(q_empty + i, 1);
            mbar_init(s_full + i, 1);
            mbar_init(p_ready + 2 * i, 4);
            mbar_init(p_ready + 2 * i + 1, 4);
            mbar_init(o_full + i, 1);
            mbar_init(drain + i, 1);
            mbar_init(i_full + i, 1);
            mbar_init(i_empty + i, kItemReaders);
            mbar_init(s_free + i, 4);
            mbar_init(p_free + i, 1);
        }
        for (int i = 0; i < L::KST; ++i) {
            mbar_init(k_full + i, 1);
            mbar_init(k_empty + i, 2);
        }
        for (int i = 0; i < L::VST; ++i) {
            mbar_init(v_full + i, 1);
            mbar_init(v_empty + i, 2);
        }
        mbar_init(v_raw, 1);
        *abort_flag = *spoiled = 0;
        fence_mbar_init();
    }
    if (warp == kTmaWarp && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &map_q : lane == 1 ? &map_k : &map_v) : "memory");
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = *tmem_slot;
    const int group = p.Hq / p.Hk;
    int failed = 0;
    auto wait_for = [&](uint64_t *bar, uint32_t parity, uint32_t polls) {
        for (uint32_t i = 0; i < polls; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) break;
        }
        *abort_flag = 1;
        return false;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_for(bar, parity, kAttnPolls); };
    auto wait_copy = [&](uint64_t *bar, uint32_t parity) { return wait_for(bar, parity, p.polls); };
    // The same where the warp's lanes have to go on or stop together.
    auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    auto tile_row = [&](const Item &it, int t) { return first_row(a, it, t); };
    auto tile_blocks = [&](const Item &it, const Seq &s, int t) { return blocks_of<SPLIT>(a, it, s, t); };
    auto find_item = [&](UnitSearch &units, int k) { return item_of<SPLIT>(a, units, k); };
    // The same from the item warp, for a warp that follows them all; false when a wait gave up.
    auto see_item = [&](int k) { return wait_all(i_full + (k & 1), (k >> 1) & 1); };
    auto leave_item = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(i_empty + (k & 1));
    };
    auto take_item = [&](int k, Item &it) {
        if (!see_item(k)) return false;
        it = slots[k & 1];
        leave_item(k);
        return true;
    };
    // The softmax keeps 128 scores and what goes with them in registers: it takes some over from
    // the other warps (with 168 each some were spilled).
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (warp == kItemWarp) {
            // ---- work items, two ahead
            UnitSearch units;
            for (int k = 0;; ++k) {
                if (k >= 2 && !wait_all(i_empty + (k & 1), ((k >> 1) - 1) & 1)) {
                    failed = 1;
                    break;
                }
                const Item it = find_item(units, k);
                if (lane == 0) {
                    slots[k & 1] = it;
                    mbar_arrive(i_full + (k & 1));
                }
                __syncwarp();
                if (!it.found) break;
            }
        } else if (warp == kTmaWarp) {
            // ---- loads.  One lane issues them, so that its waits need no agreement, up to an item's last
            // values: rows behind the sequence's end are there zeroed by the whole warp.
            const uint64_t once = leave_first(), again = leave_last();
            uint32_t raw = 0;
            int nq_issued[2] = {0, 0}, nk_issued = 0, nv_issued = 0;
            bool ok = true;
            for (int k = 0; ok; ++k) {
                Item it;
                ok = take_item(k, it);
                if (!ok || !it.found) break;
                const Seq s = it.s;
                const int head0 = a.pair_heads ? 2 * it.head : it.head, kvh = head0 / group;
                const int n0 = tile_blocks(it, s, 0), n1 = tile_blocks(it, s, 1), nb = max(n0, n1), j0 = SPLIT ? it.lo : 0;
                auto load_q = [&](int t) {
                    if (nq_issued[t] > 0 && !wait(q_empty + t, (nq_issued[t] - 1) & 1)) return false;
                    mbar_arrive_expect_tx(q_full + t, L::QB);
#pragma unroll
                    for (int x = 0; x < D; x += 64)
                        tma_load_hint(sb + L::Q + t * L::QB + (x / 64) * kTile * 128, &map_q, q_full + t, x,
                                      a.pair_heads ? head0 + t : head0, s.q0 + tile_row(it, t), once);
                    ++nq_issued[t];
                    return true;
                };
                auto load_k = [&](int j) {
                    const int i = nk_issued, st = i % L::KST;
                    if (i >= L::KST && !wait(k_empty + st, (i / L::KST - 1) & 1)) return false;
                    mbar_arrive_expect_tx(k_full + st, L::KB);
#pragma unroll
                    for (int x = 0; x < D; x += 64)
                        tma_load_hint(sb + L::K + st * L::KB + (x / 64) * kTile * 128, &map_k, k_full + st, x, kvh,
                                      s.k0 + (j0 + j) * kTile, again);
                    ++nk_issued;
                    return true;
                };
                auto issue_v = [&](int j, int h, int st, uint64_t *bar) {
                    mbar_arrive_expect_tx(bar, L::VB);
#pragma unroll
                    for (int x = 0; x < DV; x += 64)
                        tma_load_hint(sb + L::V + st * L::VB + (x / 64) * L::VROWS * 128, &map_v, bar, x, kvh,
                                      s.k0 + (j0 + j) * kTile + h * L::VROWS, again);
                };
                auto v_free = [&](int st) { return nv_issued < L::VST || wait(v_empty + st, (nv_issued / L::VST - 1) & 1); };
                if (lane == 0) {
                    if (n0) ok = load_q(0);
                    if (ok && nb) ok = load_k(0);
                    if (ok && n1) ok = load_q(1);
                    for (int j = 0; j + 1 < nb && ok; ++j) {
                        ok = load_k(j + 1);
                        for (int h = 0; h < L::NV && ok; ++h) {
                            const int st = nv_issued % L::VST;
                            ok = v_free(st);
                            if (!ok) break;
                            issue_v(j, h, st, v_full + st);
                            ++nv_issued;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                nv_issued = __shfl_sync(0xffffffffu, nv_issued, 0);
                for (int h = 0; h < L::NV && nb > 0 && ok; ++h) {
                    const int st = nv_issued % L::VST;
                    const int rows = max(0, s.nk - (j0 + nb - 1) * kTile - h * L::VROWS);  // of the sequence
                    ok = __all_sync(0xffffffffu, v_free(st)) != 0;
                    if (!ok) break;
                    if (lane == 0) issue_v(nb - 1, h, st, rows < L::VROWS ? v_raw : v_full + st);
                    if (rows < L::VROWS) {
                        ok = __all_sync(0xffffffffu, wait(v_raw, raw & 1)) != 0;
                        if (!ok) mbar_wait(v_raw, raw & 1, kAttnPolls);  // the copy must still land before the CTA may end
                        ++raw;
                        if (!ok) break;
                        for (int i = lane; i < (L::VROWS - rows) * (DV / 64) * 8; i += 32) {
                            const int r = rows + i / ((DV / 64) * 8), q = i % ((DV / 64) * 8);
                            st_shared_v4(sb + L::V + st * L::VB + (q >> 3) * L::VROWS * 128 + r * 128 + (q & 7) * 16, 0, 0, 0, 0);
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(v_full + st);
                    }
                    ++nv_issued;
                }
            }
            if (!ok) failed = 1;
            // every load lands before the CTA may end
            if (lane == 0) {
                for (int t = 0; t < 2; ++t)
                    if (nq_issued[t]) mbar_wait(q_full + t, (nq_issued[t] - 1) & 1, kAttnPolls);
                for (int j = max(0, nk_issued - L::KST); j < nk_issued; ++j)
                    mbar_wait(k_full + j % L::KST, (j / L::KST) & 1, kAttnPolls);
                for (int j = max(0, nv_issued - L::VST); j < nv_issued; ++j)
                    mbar_wait(v_full + j % L::VST, (j / L::VST) & 1, kAttnPolls);
            }
            __syncwarp();
        } else {
            // ---- products of tile t.  One thread's instructions come one at a time, about five
            // cycles each, so the descriptors are bases plus constants.
            const int t = warp - kMmaWarp;
            const uint32_t id_s = idesc_bf16(kTile, kTile, false, false, p.scale < 0.f);
            const uint32_t id_o = idesc_bf16(kTile, DV, false, true);
            const uint32_t lo_kmajor = sb16 | (16u >> 4) << 16, lo_v = sb16 | (L::VROWS * 128u >> 4) << 16;
            const uint32_t q_lo = lo_kmajor + ((L::Q + t * L::QB) >> 4), t_s = tb + L::T_S + t * kTile, t_o = tb + L::T_O + t * DV,
                           t_p = tb + L::T_P + t * L::P_STEP;
            int ks = 0, vs = 0;       // ring places of the next keys and values
            uint32_t kp = 0, vp = 0;  // and the parities of their rounds
            uint32_t blocks = 0, tiles = 0;  // of this tile so far: key blocks, and items with any
            bool begun = false, ok = true;
            auto scores = [&] {
                const uint32_t k_lo = lo_kmajor + (L::K >> 4) + ks * (L::KB >> 4);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t off = ((x / 4) * kTile * 128 + (x % 4) * 32) >> 4;
                    mma_ss(t_s, desc_of(q_lo + off), desc_of(k_lo + off), id_s, x > 0);
                }
                mma_commit(s_full + t);
                mma_commit(k_empty + ks);
            };
            // A half's product with its values, the last of both of a slot letting go of it.
            auto weigh = [&](int h, int slot, bool more) {
                const uint32_t v_lo = lo_v + (L::V >> 4) + slot * (L::VB >> 4) + (L::NV == 1 ? h * 4 * (2048 >> 4) : 0);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mma_ts(t_o, t_p + (4 * h + x) * 8, desc_of(v_lo + x * (2048 >> 4)), id_o, x > 0 ? 1u : more);
                if (L::NV == 2 || h == 1) mma_commit(v_empty + slot);
            };
            // With weights of their own each tile's products go ahead as their operands come: the scores of
            // block j + 1, then the product of block j.
            uint32_t scored = 0;  // blocks with scores so far
            for (int k = 0; L::AHEAD; ++k) {
                Item it;
                if (!ok || !take_item(k, it)) {
                    failed = 1;
                    break;
                }
                if (!it.found) break;
                const int n0 = tile_blocks(it, it.s, 0), n1 = tile_blocks(it, it.s, 1), nb = max(n0, n1), nt = t ? n1 : n0;
                if (nt) ok = wait_copy(q_full + t, tiles & 1);
                for (int j = -1; j < nb; ++j) {
                    if (j + 1 < nb) {
                        const bool mine = j + 1 < nt;
                        ok = ok && wait(k_full + ks, kp);
                        if (mine && scored > 0) ok = ok && wait(s_free + t, (scored - 1) & 1);
                        fence_after_sync();
                        if (elect_one() && ok) {
                            if (mine) {
                                scores();
                                if (j + 2 == nt) mma_commit(q_empty + t);
                            } else {
                                mbar_arrive(k_empty + ks);  // every block is let go of by both tiles
                            }
                        }
                        __syncwarp();
                        scored += mine;
                        if (++ks == L::KST) ks = 0, kp ^= 1;
                    }
                    if (j < 0) continue;
                    const bool mine = j < nt;
                    ok = ok && wait(v_full + vs, vp);
                    if (mine) ok = ok && wait(p_ready + 2 * t, (blocks + j) & 1);
                    fence_after_sync();
                    if (mine && elect_one() && ok) weigh(0, vs, j > 0);
                    __syncwarp();
                    if (mine) ok = ok && wait(p_ready + 2 * t + 1, (blocks + j) & 1);
                    fence_after_sync();
                    if (elect_one() && ok) {
                        if (mine) {
                            weigh(1, vs, true);
                            mma_commit(p_free + t);
                            if (j + 1 == nt) mma_commit(o_full + t);
                        } else {
                            mbar_arrive(v_empty + vs);
                        }
                    }
                    __syncwarp();
                    if (++vs == L::VST) vs = 0, vp ^= 1;
                }
                blocks += nt;
                tiles += nt > 0;
                ok = __all_sync(0xffffffffu, ok);
            }
            for (int k = 0; !L::AHEAD; ++k) {
                Item it;
                // both product warps go on or stop together: each waits for the other's turns
                const bool taken = take_item(k, it);
                if (pair_any(3, !ok || !taken)) {
                    failed = 1;
                    break;
                }
                if (!it.found) break;
                const Seq s = it.s;
                const int n0 = tile_blocks(it, s, 0), n1 = tile_blocks(it, s, 1), nb = max(n0, n1), nt = t ? n1 : n0;
                auto next_keys = [&] {
                    if (++ks == L::KST) ks = 0, kp ^= 1;
                };
                if (nt) ok = wait_copy(q_full + t, tiles & 1);
                if (nb) {
                    ok = ok && wait(k_full + ks, kp);
                    fence_after_sync();
                    if (elect_one() && ok) {
                        if (nt) {
                            scores();
                            if (nt == 1) mma_commit(q_empty + t);
                        } else {
                            mbar_arrive(k_empty + ks);  // every block is let go of by both tiles
                        }
                    }
                    next_keys();
                }
                for (int j = 0; j < nb; ++j) {
                    const bool mine = j < nt, next = j + 1 < nt, more = j + 1 < nb;  // (an idle tile follows the rings too)
                    ok = ok && wait(v_full + vs, vp);
                    if (more) ok = ok && wait(k_full + ks, kp);
                    if (mine) ok = ok && wait(p_ready + 2 * t, (blocks + j) & 1);
                    fence_after_sync();
                    if (t || begun) turn_wait(1 + t);
                    begun = true;
                    if (mine && elect_one() && ok) weigh(0, vs, j > 0);
                    __syncwarp();
                    const int vs0 = vs;
                    if (L::NV == 2) {
                        if (!mine && ok && lane == 0) mbar_arrive(v_empty + vs0);
                        if (++vs == L::VST) vs = 0, vp ^= 1;
                        ok = ok && wait(v_full + vs, vp);
                    }
                    if (mine) ok = ok && wait(p_ready + 2 * t + 1, (blocks + j) & 1);
                    fence_after_sync();
                    if (elect_one() && ok) {
                        if (mine) {
                            weigh(1, vs, true);
                            // the next scores overwrite this block's weights: behind the product in the same queue
                            if (next) {
                                scores();
                                if (j + 2 == nt) mma_commit(q_empty + t);
                            } else {
                                mma_commit(o_full + t);
                            }
                        } else {
                            mbar_arrive(v_empty + vs);
                        }
                        if (!next && more) mbar_arrive(k_empty + ks);
                    }
                    __syncwarp();
                    turn_pass(2 - t);
                    if (more) next_keys();
                    if (++vs == L::VST) vs = 0, vp ^= 1;
                }
                blocks += nt;
                tiles += nt > 0;
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!t && begun) turn_wait(1);  // the other warp's last turn was passed here
            // nothing issued may still run, and no commit arrive, once the CTA has ended
            if (elect_one()) {
                mma_commit(drain + t);
                mbar_wait(drain + t, 0, kAttnPolls);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // ---- softmax of tile t, a thread per row
        const int t = warp >> 2, m_row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tb + lane_base + L::T_S + t * kTile, t_o = tb + lane_base + L::T_O + t * DV,
                       t_p = tb + lane_base + L::T_P + t * L::P_STEP;
        const float c = fabsf(p.scale) * kLog2e;
        uint32_t blocks = 0, tiles = 0;  // of this tile so far: key blocks, and items with any
        bool ok = see_item(0);
        int k = 0;
        for (; ok && slots[k & 1].found; ++k) {
            int nt, seen, seen_first;  // what the loop over the keys needs of the item; the rest is read again behind it
            {
                const Item it = slots[k & 1];
                const int row0 = tile_row(it, t), row = row0 + m_row, more = it.s.nk - it.s.nq;
                nt = tile_blocks(it, it.s, t);
                seen = max(0, min(it.s.nk, row + 1 + more));
                seen_first = max(0, min(it.s.nk, row0 + 1 + more));  // of the tile's first row
                if (SPLIT) seen -= it.lo * kTile, seen_first -= it.lo * kTile;  // keys of this part
            }
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < nt && ok; ++j, ++blocks) {
                ok = wait_all(s_full + t, blocks & 1);
                if (!ok) break;
                fence_after_sync();
                float x[128];
#pragma unroll
                for (int i = 0; i < 128; i += 32) tmem_ld32(t_s + i, x + i);
                wait_ld64(x);
                wait_ld64(x + 64);
                if (L::AHEAD) {
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free + t);
                }
                if ((j + 1) * kTile > seen_first) {
                    // keys behind what the row sees, by runs of 32: those that the warp's first row sees whole
                    // need no look
                    const int lim = seen - j * kTile, w_lo = __shfl_sync(0xffffffffu, lim, 0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (32 * q + 32 <= w_lo) continue;
#pragma unroll
                        for (int i = 32 * q; i < 32 * q + 32; ++i)
                            if (i >= lim) x[i] = -INFINITY;
                    }
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int i = 4; i < 124; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(fmaxf(mx[e], x[i + e]), x[i + 4 + e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[124 + e]);
                const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool raise = mb > m + kSlack;
                if (L::AHEAD && blocks > 0) {  // the last weights, and the products that O is to hold
                    ok = wait_all(p_free + t, (blocks - 1) & 1);
                    fence_after_sync();
                }
                if (__any_sync(0xffffffffu, raise)) {
                    const float f = raise ? ex2(m - mb) : 1.f;
                    if (raise) m = mb;
                    l *= f;
                    if (j > 0) {  // the products before are done: (AHEAD) waited for, else said by the scores' arrival
#pragma unroll 1
                        for (int d = 0; d < DV; d += 16) {
                            uint32_t o[16];
                            tmem_ld16(t_o + d, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(t_o + d, o);
                        }
                    }
                }
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                weights32(x, c, m, sum);
                weights32(x + 32, c, m, sum);
                tmem_st16x2(t_p, x, x + 32);
                weights32(x + 64, c, m, sum);
                hand_over(p_ready + 2 * t);
                weights32(x + 96, c, m, sum);
                tmem_st16x2(t_p + 32, x + 64, x + 96);
                hand_over(p_ready + 2 * t + 1);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            // What does not need O comes before the wait for it: the next item, the row's factor and places.
            const Item it = slots[k & 1];
            const Seq s = it.s;
            const int row0 = tile_row(it, t), row = row0 + m_row, head = a.pair_heads ? 2 * it.head + t : it.head;
            leave_item(k);
            const bool more = !ok || see_item(k + 1);
            const bool live = row < s.nq;
            const int64_t out = (int64_t)(s.q0 + row) * p.Hq + head;
            float inv = SPLIT ? 1.f : l == 0.f ? 0.f : 1.f / l, lse = l == 0.f ? -INFINITY : (log2f(l) + m) * kLn2;
            // Four lanes exchange 16-byte pieces of their rows, so that they write 64 bytes of a row
            // together (lanes writing a row each touch 32 lines per store).
            const int first = row0 + (warp & 3) * 32 + (lane & ~3);  // of the four rows
            float *part = SPLIT ? a.p.ws + (int64_t)it.place * kPartFloats<DV> : nullptr;
            const bool bf16 = !SPLIT && p.o_bf16;
            const int esz = bf16 ? 2 : 4;
            uint8_t *o_rows = SPLIT ? reinterpret_cast<uint8_t *>(part + (t * kTile + first - row0) * DV) + (lane & 3) * 16
                                    : static_cast<uint8_t *>(p.o) + ((int64_t)(s.q0 + first) * p.Hq + head) * DV * esz + (lane & 3) * 16;
            const int64_t pitch = (int64_t)(SPLIT ? 1 : p.Hq) * DV * esz;
            if (ok && nt > 0) ok = wait_all(o_full + t, tiles & 1);
            tiles += nt > 0;
            fence_after_sync();
            if (!ok) inv = lse = l = __int_as_float(0x7fc00000);
            if (row0 + (warp & 3) * 32 < s.nq) {  // (else the warp has no such rows)
                const float2 inv2 = make_float2(inv, inv), zero = make_float2(0.f, 0.f);
                float2 odd[4] = {zero, zero, zero, zero};  // 0, or NaN where an output is not finite
#pragma unroll 1
                for (int d = SPLIT && nt == 0 ? DV : 0; d < DV; d += 64) {
                    float r[64];
                    if (ok && nt > 0) {
                        tmem_ld32(t_o + d, r);
                        tmem_ld32(t_o + d + 32, r + 32);
                        wait_ld64(r);
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i) r[i] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float2 x = fma2(make_float2(r[2 * i], r[2 * i + 1]), inv2, zero);
                        odd[i & 3] = fma2(x, zero, odd[i & 3]);
                        r[2 * i] = x.x;
                        r[2 * i + 1] = x.y;
                    }
                    auto store = [&](uint32_t (&w)[16], int byte) {
                        transpose_quad(w);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (first + i < s.nq) {
                                const uint4 x = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                                uint4 *at = reinterpret_cast<uint4 *>(o_rows + i * pitch + byte);
                                if (SPLIT)
                                    *at = x;
                                else
                                    __stcs(at, x);
                            }
                    };
                    uint32_t w[16];
                    if (bf16) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(r[32 * h + 2 * i], r[32 * h + 2 * i + 1]);
                            store(w, (d + 32 * h) * 2);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(r[16 * h + i]);
                            store(w, (d + 16 * h) * 4);
                        }
                    }
                }
                __syncwarp();
                if (live) {
                    if (SPLIT) {
                        part[2 * kTile * DV + t * kTile + m_row] = m;
                        part[2 * kTile * (DV + 1) + t * kTile + m_row] = l;
                    } else if (p.lse) {
                        p.lse[out] = lse;
                    }
                    const float2 any = add2(add2(odd[0], odd[1]), add2(odd[2], odd[3]));
                    if (isnan(any.x + any.y)) *spoiled = 1;
                }
            }
            ok = ok && more;
        }
        if (!ok) {  // what this CTA still had to do: NaN
            failed = 1;
            UnitSearch units;
            for (;; ++k) {
                const Item it = find_item(units, k);
                if (!it.found) break;
                const Seq s = it.s;
                const int row = tile_row(it, t) + m_row, head = a.pair_heads ? 2 * it.head + t : it.head;
                if (row >= s.nq) continue;
                if (SPLIT) {
                    float *part = a.p.ws + (int64_t)it.place * kPartFloats<DV> + 2 * kTile * DV + t * kTile + m_row;
                    part[0] = 0.f;
                    part[2 * kTile] = __int_as_float(0x7fc00000);
                    continue;
                }
                const int64_t out = (int64_t)(s.q0 + row) * p.Hq + head;
                for (int d = 0; d < DV; ++d) st_out(p.o, out * DV + d, __int_as_float(0x7fc00000), p.o_bf16);
                if (p.lse) p.lse[out] = __int_as_float(0x7fc00000);
            }
        }
    }
    fence_before_sync();
    const bool gave_up = __syncthreads_or(failed);
    if (gave_up && threadIdx.x == 0) atomicAdd(&g_attn_prompt_timeouts, 1);
    fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(tb, 512);
    // Here no warp waits for another any more, however many keys such a row sees.
    if (warp < kMmaWarp && !gave_up && *spoiled) rescue_rows<D, DV, SPLIT>(a);
}

// Joins the parts of a unit and head: `rows` of their 2 x 128 rows a CTA, four channels a thread;
// four parts are on their way at a time (one after the other, 8 parts took 15 us).
constexpr int kJoinThreads = 256;
template <int DV>
__global__ void __launch_bounds__(kJoinThreads) attn_prompt_join_kernel(const __grid_constant__ Args a, int rows) {
    const PromptParams &p = a.p;
    __shared__ Seq s_seq;
    __shared__ int s_row0;  // or -1
    const int unit = blockIdx.x / a.n_heads, pair = blockIdx.x % a.n_heads;
    if (threadIdx.x < 32) {
        UnitSearch units;
        int seq = 0, row0 = 0;
        const bool found = units.find(p, a.pair_heads ? 7 : 8, unit, seq, row0);
        const Seq s = seq_of(p, seq);
        if (threadIdx.x == 0) {
            s_seq = s;
            s_row0 = found ? row0 : -1;
        }
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (s_row0 < 0) return;
    constexpr int LANES = DV / 4;  // of a row
    const int d = threadIdx.x % LANES * 4;
    const float *part = p.ws + (int64_t)blockIdx.x * a.parts * kPartFloats<DV>;
    for (int r0 = 0; r0 < rows; r0 += kJoinThreads / LANES) {
        const int r = blockIdx.y * rows + r0 + threadIdx.x / LANES, t = r / kTile;
        const int row = s_row0 + (a.pair_heads ? r % kTile : r), head = a.pair_heads ? 2 * pair + t : pair;
        if (row >= s_seq.nq) continue;
        float M = -INFINITY, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < a.parts; i0 += 4) {
            float m[4], l[4];
            float4 y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *x = part + (int64_t)(i0 + i) * kPartFloats<DV>;
                const bool is = i0 + i < a.parts;
                m[i] = is ? __ldcg(x + 2 * kTile * DV + r) : -INFINITY;
                l[i] = is ? __ldcg(x + 2 * kTile * (DV + 1) + r) : 0.f;
                y[i] = is ? __ldcg(reinterpret_cast<const float4 *>(x + r * DV + d)) : o;
            }
            const float next = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), M);
            const float g = M == -INFINITY ? 1.f : ex2(M - next);  // (all zero so far)
            M = next;
            L *= g;
            o = make_float4(o.x * g, o.y * g, o.z * g, o.w * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (l[i] == 0.f) continue;  // the part saw nothing, and may have left no O
                const float f = ex2(m[i] - M);
                L = fmaf(l[i], f, L);
                o.x = fmaf(y[i].x, f, o.x);
                o.y = fmaf(y[i].y, f, o.y);
                o.z = fmaf(y[i].z, f, o.z);
                o.w = fmaf(y[i].w, f, o.w);
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int64_t out = (int64_t)(s_seq.q0 + row) * p.Hq + head;
        if (p.o_bf16)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + out * DV + d) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + out * DV + d) =
                make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (p.lse && d == 0) p.lse[out] = L == 0.f ? -INFINITY : (log2f(L) + M) * kLn2;
    }
}

// A tensor of rows (heads of `dim` bf16 elements, `stride` elements from row to row) in boxes
// of 64 channels x 1 head x box_rows.
bool encode(chunk::EncodeTiledFn enc, CUtensorMap *map, const void *base, int dim, int heads, int64_t rows,
            int64_t stride, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) set_error("attn_prompt: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return r == CUDA_SUCCESS;
}

struct Shape {
    int pair_heads, n_heads, parts;
    int64_t units;  // at most: a sequence of n rows has at most n / rows + 1
};

// Work items of a call, and how many share the keys of a unit and head.  With few units the
// longest alone would set the time, and most SMs would idle.  A part costs an item's beginning and
// end (about 2.5 blocks of 128 keys), the joining launch (3.5), and its sums' way through L2 (0.012
// for each part of the call).  The number of parts with the least estimate for sequences of equal
// lengths is taken, for at most three items an SM.  Channels 128, whole and in parts:
// 2 heads over one key head, 1024 tokens 16.8 and 12.2 us, 8192 tokens 88 and 36 us; 128 queries
// over 4096 keys with 32/8 heads 48 and 18 us; 16/4 heads over 2048 tokens 27.7 and 30.8 us, which
// the estimate leaves whole.
Shape shape_of(int64_t Tq, int64_t Tk, int N, int Hq, int Hk) {
    Shape x;
    x.pair_heads = (Hq / Hk) % 2 == 0;
    x.n_heads = x.pair_heads ? Hq / 2 : Hq;
    x.parts = 1;
    const int rows = x.pair_heads ? kTile : 2 * kTile, sms = sm_count();
    x.units = Tq / rows + N;
    const int64_t q = Tq / N, k = Tk / N, per = (q + rows - 1) / rows, items = per * N * x.n_heads;
    if (items * 2 > 3 * sms || k <= kTile) return x;
    double total = 0, best = 0;  // in key blocks
    int64_t longest = 0;
    for (int64_t u = 0; u < per; ++u) {
        const int64_t seen = std::min(q, (u + 1) * rows) + k - q, n = seen > 0 ? (seen + kTile - 1) / kTile : 0;
        total += (double)n * N * x.n_heads;
        longest = std::max(longest, n);
    }
    for (int s = 1; s <= 32 && s <= longest && (s == 1 || x.units * x.n_heads * s <= 3 * sms); ++s) {
        const int64_t rounds = (items * s + sms - 1) / sms;
        const double run = std::max((double)((longest + s - 1) / s), (rounds > 1 ? 1.2 : 1.0) * total / sms);
        const double t = 2.5 * rounds + run + (s > 1 ? 3.5 + 0.012 * items * s : 0.0);
        if (s == 1 || t < best) best = t, x.parts = s;
    }
    return x;
}

template <int D, int DV, bool SPLIT>
kda_status launch(const PromptParams &p, const Shape &shape, cudaStream_t st) {
    using L = Cfg<D, DV>;
    chunk::EncodeTiledFn enc = reinterpret_cast<chunk::EncodeTiledFn>(tensor_map_encoder());
    if (!enc) {
        set_error("attn_prompt: cuTensorMapEncodeTiled is not available from the driver");
        return KDA_ERR_CUDA;
    }
    static DeviceOnce configured;
    const int dev = current_device();
    const auto kernel = attn_prompt_kernel<D, DV, SPLIT>;
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM) != cudaSuccess) {
            set_error("attn_prompt: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        cudaFuncAttributes attr;
        if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess || attr.numRegs < kLaunchRegs) {
            cudaGetLastError();
            set_error("attn_prompt: built with fewer registers than its warps share out");
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    CUtensorMap mq, mk, mv;
    // without keys nothing is loaded; the map still needs an address
    const bool keys = p.Tk > 0;
    if (!encode(enc, &mq, p.q, D, p.Hq, p.Tq, p.q_stride, kTile) ||
        !encode(enc, &mk, keys ? p.k : p.q, D, keys ? p.Hk : p.Hq, keys ? p.Tk : p.Tq, keys ? p.k_stride : p.q_stride, kTile) ||
        !encode(enc, &mv, keys ? p.v : p.q, keys ? DV : D, keys ? p.Hk : p.Hq, keys ? p.Tk : p.Tq,
                keys ? p.v_stride : p.q_stride, L::VROWS))
        return KDA_ERR_CUDA;
    Args a;
    memset(&a, 0, sizeof(a));
    a.p = p;
    a.pair_heads = shape.pair_heads;
    a.n_heads = shape.n_heads;
    a.parts = SPLIT ? shape.parts : 1;
    const int64_t items = shape.units * a.n_heads * a.parts;
    if (items > INT32_MAX) {
        set_error("kda_attn_prompt: too many tokens");
        return KDA_ERR_UNSUPPORTED;
    }
    a.items = (int)items;
    const int sms = sm_count();
    kernel<<<a.items < sms ? a.items : sms, kThreads, L::SMEM, st>>>(mq, mk, mv, a);
    note_launch();
    const kda_status s = check_launch("attn_prompt_kernel");
    if (!SPLIT || s != KDA_OK) return s;
    cudaLaunchConfig_t cfg = {};
    int rows = kJoinThreads / (DV / 4);  // more where that would be many waves of CTAs
    while (rows < 64 && (int64_t)(a.items / a.parts) * (2 * kTile / rows) > 8 * sms) rows *= 2;
    cfg.gridDim = dim3(a.items / a.parts, 2 * kTile / rows);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // starts while the first kernel ends; waits for it before it reads
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_prompt_join_kernel<DV>, a, rows);
    note_launch();
    if (e != cudaSuccess) {
        set_error("attn_prompt_join_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return check_launch("attn_prompt_join_kernel");
}

template <int D, int DV>
kda_status run(const PromptParams &p, cudaStream_t st) {
    const Shape shape = shape_of(p.Tq, p.Tk, p.N, p.Hq, p.Hk);
    return p.ws && shape.parts > 1 ? launch<D, DV, true>(p, shape, st) : launch<D, DV, false>(p, shape, st);
}

}  // namespace

int take_attn_prompt_timeouts(cudaStream_t st) {
    int n = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&n, g_attn_prompt_timeouts, sizeof(int), 0, cudaMemcpyDeviceToHost, st) !=
            cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_attn_prompt_timeouts, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) !=
            cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        set_error("attn_prompt: cannot read the timeout counter: %s", cudaGetErrorString(cudaGetLastError()));
        return -1;
    }
    return n;
}

size_t attn_prompt_workspace_bytes(int64_t Tq, int64_t Tk, int N, int Hq, int Hk, int DV) {
    const Shape x = shape_of(Tq, Tk, N, Hq, Hk);
    return x.parts == 1 ? 0 : (size_t)(x.units * x.n_heads * x.parts) * (2 * kTile * (DV + 2)) * sizeof(float);
}

kda_status launch_attn_prompt(const PromptParams &p, cudaStream_t st) {
    if (p.Tq == 0) return KDA_OK;
    if (p.D == 64) return run<64, 64>(p, st);
    if (p.D == 128) return run<128, 128>(p, st);
    return run<192, 128>(p, st);
}

}  // namespace kda
