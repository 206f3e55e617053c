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
// row's 64 weights are one swizzled 128-byte line.  Queries (72 KB) and two steps of the
// cache (144 KB) fill the shared memory, which is what limits a tile to 64 rows.
//
// The cache arrives by TMA in a ring of 128-channel units (the shared channels in one of their own),
// and a unit is free again when the one product of O^T that reads it is through.  A step's
// scores are formed while the softmax works on the last step's.  The softmax's reference moves only where a row's maximum rises by more than
// 2^kSlack, since moving it means rescaling O^T in TMEM.
//
// Work split.  All steps of all units (a sequence's groups of `G` tiles, each tile on a CTA of
// its own, so that the G read the same tokens at about the same time) are numbered in one line,
// kPad places before each unit standing for what it costs beside its steps; the line is cut into
// equal pieces.  Units that more than one CTA took leave their sums in a workspace, and
// attn_latent_join_kernel adds them in their order, so results do not depend on timing.
#include <cuda.h>

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
constexpr int kSoftWarps = 4, kMmaWarp = 4, kLoadWarp = 5;
constexpr int kThreads = 192;
constexpr int kSlots = 4;               // work items under way
constexpr int kPad = 4;                 // a unit's own cost in steps
constexpr int kMinPiece = 6;            // places of a CTA at least
constexpr int kMaxUnits = 12, kMaxShared = 4;  // ring places at most
constexpr uint32_t kUnitBytes = kStep * 256, kSharedBytes = kStep * 128;
constexpr uint32_t kTmemO = 2 * kStep;  // TMEM columns: scores of two steps, then O^T
constexpr float kSlack = 8.f;           // log2: how far a score may exceed the reference
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNaN = __builtin_nanf("");
constexpr int kMaxSmem = 232448;
constexpr uint32_t kProductPolls = 1u << 27;  // of the products' warp, which looks without waiting: seconds

__device__ int g_attn_latent_timeouts = 0;

struct Plan {
    int hp, tk;       // heads (a multiple of 8) and tokens of a tile: hp * tk rows
    int parts;        // tiles that share a token's heads
    int G;            // tiles of a unit
    int pieces;       // of the line
    int cut;          // units may be cut; else each lies in the piece where it begins
    int n;            // rows of a tile as the products' N: hp * tk, a multiple of 16
    int units, shared;  // ring places
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
    uint64_t q_full, q_empty, o_free, p_ready, p_free, drain;
    uint64_t s_full[2], s_free[2];
    uint64_t i_full[kSlots], i_empty[kSlots];
    uint64_t u_full[kMaxUnits], u_empty[kMaxUnits];
    uint64_t r_full[kMaxShared], r_empty[kMaxShared];
    Item slots[kSlots];
    int64_t row_at[kTileRows];   // a row's place in o, or -1
    float factor[kTileRows];
    int64_t scan[kThreads / 32];
    int64_t start_begin;
    int start_seq;
    uint32_t tmem;
    int abort;                   // a bounded wait gave up
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
// A 128-byte-swizzled operand's descriptor from its low word (address / 16 and leading offset);
// the row groups are 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}
// Whether a phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
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
// Units of a sequence with nq rows in the call.
__host__ __device__ __forceinline__ int64_t units_of(const Plan &pl, int64_t nq) {
    const int64_t tiles = (nq + pl.tk - 1) / pl.tk * pl.parts;
    return (tiles + pl.G - 1) / pl.G;
}
__device__ __forceinline__ int64_t places_of(const Args &a, int n) {
    int64_t t0;
    int nq;
    call_rows(a.p.cu_seqlens, a.p.tokens, n, t0, nq);
    return nq == 0 ? 0 : units_of(a.plan, nq) * (steps_of(tokens_of(a.p.c, n)) + kPad);
}

// Every thread's share of the sequences measured: the line's length, and where the share begins.
struct Line {
    int64_t total, mine;
    int first, last;
};
__device__ __forceinline__ Line measure_line(const Args &a, int64_t *scan, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.p.c.N, per = (N + threads - 1) / threads;
    Line l;
    l.first = min(tid * per, N);
    l.last = min(l.first + per, N);
    int64_t own = 0;
    for (int n = l.first; n < l.last; ++n) own += places_of(a, n);
    int64_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    l.mine = x - own;
    l.total = 0;
    for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) l.mine += scan[w];
        l.total += scan[w];
    }
    return l;
}
__host__ __device__ __forceinline__ int64_t piece_places(int64_t total, int pieces) { return (total + pieces - 1) / pieces; }

// A tile's rows and what they see.
struct Tile {
    int t0, tokens, head0, seen0, steps;
};
__device__ __forceinline__ Tile tile_of(const Plan &pl, int64_t t0, int nq, int len, int64_t r) {
    const int64_t i0 = r / pl.parts * pl.tk;
    Tile t;
    t.head0 = (int)(r % pl.parts) * pl.hp;
    t.tokens = (int)max((int64_t)0, min((int64_t)pl.tk, nq - i0));
    t.t0 = (int)(t0 + i0);
    t.seen0 = (int)(len - nq + i0 + 1);
    t.steps = t.tokens > 0 ? steps_of(max(0, t.seen0 + t.tokens - 1)) : 0;
    return t;
}
__device__ __forceinline__ int64_t part_floats(const Plan &pl) { return (int64_t)pl.hp * pl.tk * (kLatent + 2); }

// Goes through the work items of one tile place `g` of a piece.
struct Walk {
    int64_t L0, L1, begin, u, units;  // the piece, the next unit's place on the line, its number in its sequence
    int n, nq, len;
    int64_t t0;
    __device__ void open(const Args &a) {  // the sequence n, or the next one with rows
        for (;; ++n) {
            if (n >= a.p.c.N) return;
            call_rows(a.p.cu_seqlens, a.p.tokens, n, t0, nq);
            if (nq > 0) break;
        }
        len = tokens_of(a.p.c, n);
        units = units_of(a.plan, nq);
    }
    __device__ void start(const Args &a, int64_t l0, int64_t l1, int seq, int64_t seq_begin) {
        L0 = l0;
        L1 = l1;
        n = seq;
        if (n < 0) {
            n = a.p.c.N;
            return;
        }
        open(a);
        const int64_t per = steps_of(len) + kPad;
        u = (l0 - seq_begin) / per;
        begin = seq_begin + u * per;
    }
    __device__ Item next(const Args &a, int piece, int g) {
        const Plan &pl = a.plan;
        Item it;
        it.found = 0;
        it.bad = 0;
        while (n < a.p.c.N && begin < L1) {
            const int steps = steps_of(len);
            const int64_t first = begin + kPad, at = begin;
            const Tile t = tile_of(pl, t0, nq, len, u * pl.G + g);
            it.seq = n;
            begin += steps + kPad;
            if (++u == units) {
                ++n;
                u = 0;
                open(a);
            }
            if (t.tokens == 0) continue;
            it.t0 = t.t0;
            it.tokens = t.tokens;
            it.head0 = t.head0;
            it.seen0 = t.seen0;
            it.part = -1;
            if (!pl.cut || t.steps == 0) {
                if (at < L0) continue;
                it.s0 = 0;
                it.s1 = t.steps;
            } else {
                it.s0 = (int)max(L0 - first, (int64_t)0);
                it.s1 = (int)min(L1 - first, (int64_t)t.steps);
                if (it.s0 >= it.s1) continue;
                if (it.s0 > 0 || it.s1 < t.steps)
                    it.part = (((int64_t)piece * pl.G + g) * 2 + (it.s0 > 0 ? 0 : 1)) * part_floats(pl);
            }
            it.found = 1;
            return it;
        }
        return it;
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    attn_latent_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c,
                       const __grid_constant__ Args a) {
    const AttnLatentParams &p = a.p;
    const Plan &pl = a.plan;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm), sb16 = sb >> 4;
    Bars &b = *reinterpret_cast<Bars *>(sm + pl.at_bars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int piece = blockIdx.x / pl.G, g = blockIdx.x - piece * pl.G;
    const uint32_t q_rows = pl.hp * pl.tk;
    volatile int *abort_flag = &b.abort;

    if (pl.cut) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        mbar_init(&b.q_full, 1);
        mbar_init(&b.q_empty, 1);
        mbar_init(&b.o_free, kSoftWarps);
        mbar_init(&b.p_ready, kSoftWarps);
        mbar_init(&b.p_free, 1);
        mbar_init(&b.drain, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(b.s_full + i, 1);
            mbar_init(b.s_free + i, kSoftWarps);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(b.i_full + i, 1);
            mbar_init(b.i_empty + i, kSoftWarps + 1);
        }
        for (int i = 0; i < pl.units; ++i) {
            mbar_init(b.u_full + i, 1);
            mbar_init(b.u_empty + i, 1);
        }
        for (int i = 0; i < pl.shared; ++i) {
            mbar_init(b.r_full + i, 1);
            mbar_init(b.r_empty + i, 1);
        }
        b.abort = 0;
        b.start_seq = -1;
        fence_mbar_init();
    }
    if (warp == kLoadWarp && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &map_q : &map_c) : "memory");
    if (warp == kMmaWarp) {
        tmem_alloc(&b.tmem, 512);
        tmem_relinquish();
    }
    const Line line = measure_line(a, b.scan, kThreads);  // (a barrier inside)
    const int64_t S = piece_places(line.total, pl.pieces), L0 = piece * S, L1 = min(L0 + S, line.total);
    {
        int64_t at = line.mine;
        for (int n = line.first; n < line.last; ++n) {
            const int64_t pn = places_of(a, n);
            if (L0 >= at && L0 < at + pn && L0 < L1) {
                b.start_seq = n;
                b.start_begin = at;
            }
            at += pn;
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tb = b.tmem;
    auto wait_for = [&](uint64_t *bar, uint32_t parity, uint32_t polls) {
        for (uint32_t i = 0; i < polls; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) break;
        }
        *abort_flag = 1;
        return false;
    };
    // All lanes of a warp go on or stop together.
    auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar, parity, kAttnPolls)) != 0; };
    auto wait_copy = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_for(bar, parity, p.polls)) != 0; };

    if (warp == kLoadWarp) {
        // ---- work items, and the copies
        Walk w;
        w.start(a, L0, L1, b.start_seq, b.start_begin);
        uint32_t nu = 0, nr = 0, nq = 0;   // units, shared units and query tiles so far
        uint32_t us = 0, up = 1, rs = 0, rp = 1;  // ring places, and the parity of the wait for them
        bool ok = true;
        const int sub = min(kStep, p.c.P);  // rows of a copy
        for (uint32_t k = 0; ok; ++k) {
            const Item it = w.next(a, piece, g);
            const int slot = k % kSlots;
            if (k >= kSlots) ok = wait(b.i_empty + slot, (k / kSlots - 1) & 1);
            if (!ok) break;
            if (lane == 0) {
                b.slots[slot] = it;
                mbar_arrive(b.i_full + slot);
            }
            __syncwarp();
            if (!it.found) break;
            if (it.s0 == it.s1) continue;
            if (nq > 0) ok = wait(&b.q_empty, (nq - 1) & 1);
            if (!ok) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&b.q_full, 9 * q_rows * 128);
                for (int x = 0; x < 9; ++x)
                    tma_load_3d(sb + x * q_rows * 128, &map_q, &b.q_full, x * 64, it.head0, it.t0);
            }
            ++nq;
            const int last = min(it.seen0 + it.tokens - 1, it.s1 * kStep);  // tokens that the tile needs
            const int per_step = kStep / sub, subs = (last + sub - 1) / sub;
            const int32_t *table = p.c.block_table + (int64_t)it.seq * p.c.max_blocks;
            const int in_page = p.c.p_shift - (sub == 16 ? 4 : sub == 32 ? 5 : 6);  // log2 of a page's copies
            int base = it.s0 * per_step, pages = -1, more = -1;  // pages of copies base + lane, and of the 32 behind them
            auto fetch = [&](int i) { return i < subs ? __ldg(table + (i >> in_page)) : -1; };
            pages = fetch(base + lane);
            more = fetch(base + 32 + lane);
            for (int s = it.s0; s < it.s1 && ok; ++s) {
                int at[4], n_sub = 0;  // rows of the cache, -1: nothing to copy
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    at[j] = -1;
                    if (j >= per_step) continue;
                    const int i = s * per_step + j;
                    if (i - base >= 32) {
                        base += 32;
                        pages = more;
                        more = fetch(base + 32 + lane);
                    }
                    const int page = __shfl_sync(0xffffffffu, pages, i - base);
                    if (i >= subs) continue;
                    if ((uint32_t)page >= (uint32_t)p.c.n_pages) {
                        if (lane == 0) *(volatile int *)&b.slots[slot].bad = 1;
                        continue;
                    }
                    at[j] = (page << p.c.p_shift) + ((i << (p.c.p_shift - in_page)) & (p.c.P - 1));
                    ++n_sub;
                }
                __syncwarp();
                // the shared channels first: their scores come first
                ok = nr < (uint32_t)pl.shared || wait(b.r_empty + rs, rp);
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(b.r_full + rs, n_sub * sub * 128);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (at[j] >= 0)
                            tma_load_2d(sb + pl.at_shared + rs * kSharedBytes + j * sub * 128, &map_c, b.r_full + rs, kLatent, at[j]);
                }
                __syncwarp();
                ++nr;
                if (++rs == (uint32_t)pl.shared) rs = 0, rp ^= 1;
                for (int m = 0; m < 4; ++m) {
                    ok = nu < (uint32_t)pl.units || wait(b.u_empty + us, up);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(b.u_full + us, n_sub * sub * 256);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (at[j] >= 0)
                                for (int h = 0; h < 2; ++h)
                                    tma_load_2d(sb + pl.at_units + us * kUnitBytes + h * kSharedBytes + j * sub * 128, &map_c,
                                                b.u_full + us, m * 128 + h * 64, at[j]);
                    }
                    __syncwarp();
                    ++nu;
                    if (++us == (uint32_t)pl.units) us = 0, up ^= 1;
                }
            }
        }
        // every copy lands before the CTA may end
        if (lane == 0) {
            if (nq) mbar_wait(&b.q_full, (nq - 1) & 1, kAttnPolls);
            for (uint32_t j = nr > (uint32_t)pl.shared ? nr - pl.shared : 0; j < nr; ++j)
                mbar_wait(b.r_full + j % pl.shared, (j / pl.shared) & 1, kAttnPolls);
            for (uint32_t j = nu > (uint32_t)pl.units ? nu - pl.units : 0; j < nu; ++j)
                mbar_wait(b.u_full + j % pl.units, (j / pl.units) & 1, kAttnPolls);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---- products
        const uint32_t id_s = idesc_bf16(64, kStep, false, false, p.scale < 0.f);
        const uint32_t id_o = idesc_bf16(128, pl.n, true, false);
        const uint32_t k_major = (16u >> 4) << 16, mn_major = (kSharedBytes >> 4) << 16;
        const uint32_t q_lo = sb16 | k_major, p_lo = (sb16 + (pl.at_p >> 4)) | k_major;
        const uint32_t u_at = sb16 + (pl.at_units >> 4), r_at = sb16 + (pl.at_shared >> 4), q_chunk = q_rows * 128 >> 4;
        uint32_t us = 0, up = 0, rs = 0, rp = 0, vs = 0;  // ring places: scores' units, shared units, values' units
        uint32_t scored = 0, done = 0, items = 0;        // steps with scores, with products; items with any
        bool ok = true;
        auto ready = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0; };
        for (uint32_t k = 0; ok; ++k) {
            ok = wait(b.i_full + k % kSlots, (k / kSlots) & 1);
            if (!ok) break;
            const int found = b.slots[k % kSlots].found, nt = b.slots[k % kSlots].s1 - b.slots[k % kSlots].s0;
            __syncwarp();
            if (lane == 0) mbar_arrive(b.i_empty + k % kSlots);
            if (!found) break;
            if (nt == 0) continue;
            ok = wait_copy(&b.q_full, items & 1);
            // What is ready is issued: a step's products, or the next part of the scores of the step
            // in hand or the one behind it.  (Scores that wait for their copies must not hold up products,
            // whose units the next copies need.)
            int values = 0, scores = 0, part = 0;  // steps through; the next part, 0 being the shared channels
            uint32_t polls = 0;
            while (ok && values < nt) {
                // (the first products need the last item's output to have been read)
                if (values < scores && (values > 0 || items == 0 || ready(&b.o_free, (items - 1) & 1)) &&
                    ready(&b.p_ready, done & 1)) {
                    fence_after_sync();
                    if (elect_one()) {
                        uint32_t at = vs;
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t lo = (u_at + at * (kUnitBytes >> 4)) | mn_major;
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                mma_ss(tb + kTmemO + m * pl.n, desc_of(lo + x * (2048 >> 4)), desc_of(p_lo + 2 * x), id_o,
                                       values > 0 || x > 0);
                            mma_commit(b.u_empty + at);
                            if (++at == (uint32_t)pl.units) at = 0;
                        }
                        mma_commit(&b.p_free);
                    }
                    __syncwarp();
                    vs += 4;
                    if (vs >= (uint32_t)pl.units) vs -= pl.units;
                    ++values;
                    ++done;
                    polls = 0;
                    continue;
                }
                if (scores < nt && scores <= values + 1 && ready(part == 0 ? b.r_full + rs : b.u_full + us, part == 0 ? rp : up)) {
                    const uint32_t t_s = tb + (scored & 1) * kStep;
                    if (part == 0 && scored >= 2) {
                        ok = wait(b.s_free + (scored & 1), ((scored >> 1) - 1) & 1);
                        if (!ok) break;
                    }
                    fence_after_sync();
                    if (part == 0) {
                        if (elect_one()) {
                            const uint32_t lo = (r_at + rs * (kSharedBytes >> 4)) | k_major, ql = q_lo + 8 * q_chunk;
#pragma unroll
                            for (int x = 0; x < 4; ++x) mma_ss(t_s, desc_of(ql + 2 * x), desc_of(lo + 2 * x), id_s, x > 0);
                            mma_commit(b.r_empty + rs);
                        }
                        __syncwarp();
                        if (++rs == (uint32_t)pl.shared) rs = 0, rp ^= 1;
                        part = 1;
                    } else {
                        if (elect_one()) {
                            const uint32_t lo = (u_at + us * (kUnitBytes >> 4)) | k_major, ql = q_lo + 2 * (part - 1) * q_chunk;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
#pragma unroll
                                for (int x = 0; x < 4; ++x)
                                    mma_ss(t_s, desc_of(ql + h * q_chunk + 2 * x), desc_of(lo + h * (kSharedBytes >> 4) + 2 * x), id_s, 1);
                            if (part == 4) {
                                mma_commit(b.s_full + (scored & 1));
                                if (scores + 1 == nt) mma_commit(&b.q_empty);
                            }
                        }
                        __syncwarp();
                        if (++us == (uint32_t)pl.units) us = 0, up ^= 1;
                        if (++part == 5) part = 0, ++scores, ++scored;
                    }
                    polls = 0;
                    continue;
                }
                if (++polls > kProductPolls || __any_sync(0xffffffffu, *abort_flag)) {
                    *abort_flag = 1;
                    ok = false;
                }
            }
            ++items;
        }
        // nothing issued may still run, and no commit arrive, once the CTA has ended
        if (elect_one()) {
            mma_commit(&b.drain);
            mbar_wait(&b.drain, 0, kAttnPolls);
        }
        __syncwarp();
    } else {
        // ---- softmax, a thread per row in the lower half of each warp's lanes (where the M = 64
        // product leaves its rows), and the output, a thread per channel
        const int row = warp * 16 + (lane & 15), tok = row / pl.hp, head_in = row - tok * pl.hp;
        const bool mine = lane < 16;
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
            const bool live = mine && tok < it.tokens && head_in < pl.hp && head < p.H && row < (int)q_rows;
            const int seen = it.seen0 + tok, most = it.seen0 + it.tokens - 1;  // of this row, of the tile
            float m = -INFINITY, l = 0.f;
            for (int s = 0; s < nt; ++s, ++blocks) {
                const int j0 = (it.s0 + s) * kStep;
                ok = wait(b.s_full + (blocks & 1), (blocks >> 1) & 1);
                fence_after_sync();
                float x[kStep];
                tmem_ld32(tb + lane_base + (blocks & 1) * kStep, x);
                tmem_ld32(tb + lane_base + (blocks & 1) * kStep + 32, x + 32);
                wait_ld<kStep>(x);
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(b.s_free + (blocks & 1));
                const int lim = live ? seen - j0 : 0;
                if (j0 + kStep > it.seen0 || !live) {
#pragma unroll
                    for (int i = 0; i < kStep; ++i)
                        if (i >= lim) x[i] = -INFINITY;
                }
                float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int i = 4; i < kStep; i += 4)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[i + e]);
                const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                const bool raise = mb > m + kSlack;  // (rows that are not live: never)
                if (blocks > 0) {  // the last weights are multiplied
                    ok = ok && wait(&b.p_free, (blocks - 1) & 1);
                    fence_after_sync();
                }
                if (soft_any(raise || !ok)) {
                    if (soft_any(!ok)) {
                        ok = false;
                        break;
                    }
                    const float f = raise ? ex2(m - mb) : 1.f;
                    if (raise) m = mb;
                    l *= f;
                    if (s > 0) {
                        if (mine) b.factor[row] = f;
                        soft_sync();
                        for (int r0 = 0; r0 < pl.n; r0 += 16) {
#pragma unroll
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
                const float mm = m == -INFINITY ? 0.f : m;
                float sum[2] = {0.f, 0.f};
                uint32_t w[kStep / 2];
#pragma unroll
                for (int i = 0; i < kStep; i += 2) {
                    const float e0 = ex2(fmaf(x[i], c, -mm)), e1 = ex2(fmaf(x[i + 1], c, -mm));
                    sum[0] += e0;
                    sum[1] += e1;
                    w[i / 2] = pack_bf16x2(e0, e1);
                }
                l += sum[0] + sum[1];
                if (mine && row < pl.n) {
                    const uint32_t at = sb + pl.at_p + row * 128;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        st_shared_v4(at + ((i ^ (row & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                }
                if (j0 + kStep > it.seen0) {
                    // Tokens that not every row sees.  A weight of zero times what is not finite would not be
                    // zero: behind the tile's last token everything is cleared, and before it the rows
                    // that hold an infinity or a NaN (where a row sees one of these, its sum of weights says so).
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
            if (!ok) break;
            // ---- output
            if (nt > 0) {
                ok = wait(&b.p_free, (blocks - 1) & 1);
                fence_after_sync();
            }
            // (also: the last item's places and factors are read)
            if (soft_any(!ok)) {
                ok = false;
                break;
            }
            const bool bad = *(volatile int *)&b.slots[k % kSlots].bad != 0;
            if (bad) l = kNaN;
            const bool part = it.part >= 0;
            if (mine) {
                const int64_t out = live ? (int64_t)(it.t0 + tok) * p.H + head : -1;
                b.row_at[row] = part ? (row < (int)q_rows ? (int64_t)row : -1) : out;
                b.factor[row] = part ? 1.f : l == 0.f ? 0.f : 1.f / l;
                if (part && row < (int)q_rows) {
                    float *ml = p.ws + it.part + (int64_t)q_rows * kLatent + row;
                    ml[0] = m;
                    ml[q_rows] = l;
                }
                if (!part && live && p.lse) p.lse[out] = l == 0.f ? -INFINITY : (log2f(l) + m) * kLn2;
            }
            soft_sync();
            {
                const bool bf16 = !part && p.o_bf16;
                float *f32 = part ? p.ws + it.part : static_cast<float *>(p.o);
                for (int r0 = 0; r0 < (int)q_rows; r0 += 16)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float o[16];
                        if (nt > 0) {
                            tmem_ld16f(tb + lane_base + kTmemO + q * pl.n + r0, o);
                            wait_ld<16>(o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = 0.f;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int64_t at = b.row_at[r0 + i];
                            if (at < 0) continue;
                            const float y = o[i] * b.factor[r0 + i];
                            const int64_t e = at * kLatent + q * 128 + warp * 32 + lane;
                            if (bf16)
                                static_cast<__nv_bfloat16 *>(p.o)[e] = __float2bfloat16_rn(y);
                            else
                                f32[e] = y;
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
    if (warp == kMmaWarp) tmem_dealloc(tb, 512);
    // After a failure every row of this CTA's items becomes NaN.
    if (*abort_flag) {
        Walk w;
        w.start(a, L0, L1, b.start_seq, b.start_begin);
        for (;;) {
            const Item it = w.next(a, piece, g);
            if (!it.found) break;
            for (int i = threadIdx.x; i < (int)q_rows * kLatent; i += kThreads) {
                const int r = i / kLatent, ch = i - r * kLatent, tok = r / pl.hp, head = it.head0 + r - tok * pl.hp;
                if (it.part >= 0) {
                    p.ws[it.part + i] = kNaN;
                    if (ch < 2) p.ws[it.part + (int64_t)q_rows * (kLatent + ch) + r] = kNaN;
                } else if (tok < it.tokens && head < p.H) {
                    const int64_t out = (int64_t)(it.t0 + tok) * p.H + head;
                    st_out(p.o, out * kLatent + ch, kNaN, p.o_bf16);
                    if (ch == 0 && p.lse) p.lse[out] = kNaN;
                }
            }
        }
        if (threadIdx.x == 0) atomicAdd(&g_attn_latent_timeouts, 1);
    }
}

// Joins the tiles that more than one piece took, in the order of the pieces.  blockIdx.x is a piece
// (and a tile place of its units): the CTA looks after the unit whose first step lies in the piece
// and whose last one does not, if there is one.  gridDim.y CTAs share its rows, a row having 128 threads.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) attn_latent_join_kernel(const __grid_constant__ Args a) {
    __shared__ int64_t s_scan[kJoinThreads / 32];
    __shared__ int64_t s_begin;
    __shared__ int s_seq;
    const AttnLatentParams &p = a.p;
    const Plan &pl = a.plan;
    const int tid = threadIdx.x, piece = blockIdx.x / pl.G, g = blockIdx.x - piece * pl.G;
    const Line line = measure_line(a, s_scan, kJoinThreads);
    const int64_t S = piece_places(line.total, pl.pieces), L0 = piece * S, L1 = min(L0 + S, line.total);
    if (tid == 0) s_seq = -1;
    __syncthreads();
    if (L0 < L1) {
        int64_t at = line.mine;
        for (int n = line.first; n < line.last; ++n) {
            const int64_t pn = places_of(a, n);
            if (L1 - 1 >= at && L1 - 1 < at + pn) {
                s_seq = n;
                s_begin = at;
            }
            at += pn;
        }
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = s_seq;
    if (n < 0) return;
    int64_t t0;
    int nq;
    call_rows(p.cu_seqlens, p.tokens, n, t0, nq);
    const int len = tokens_of(p.c, n), per = steps_of(len) + kPad;
    const int64_t u = (L1 - 1 - s_begin) / per, first = s_begin + u * per + kPad;
    const Tile t = tile_of(pl, t0, nq, len, u * pl.G + g);
    if (t.steps == 0 || first < L0 || first >= L1 || first + t.steps <= L1) return;
    const int last = (int)((first + t.steps - 1) / S);  // the piece of its last step
    const int rows = pl.hp * pl.tk;
    const int64_t stride = 2 * pl.G * part_floats(pl);
    const float *ws = p.ws + ((int64_t)piece * pl.G + g) * 2 * part_floats(pl);  // slot 1 here, slot 0 of the pieces behind
    for (int r = blockIdx.y * (kJoinThreads / 128) + tid / 128; r < rows; r += gridDim.y * (kJoinThreads / 128)) {
        const int tok = r / pl.hp, head = t.head0 + r - tok * pl.hp;
        if (tok >= t.tokens || head >= p.H) continue;
        const int ch = (tid & 127) * 4;
        float m = -INFINITY, l = 0.f;
        for (int k = piece; k <= last; ++k) {
            const float *w = ws + (k - piece) * stride + (k == piece ? part_floats(pl) : 0) + (int64_t)rows * kLatent + r;
            m = fmaxf(m, __ldcg(w));
        }
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = piece; k <= last; ++k) {
            const float *w = ws + (k - piece) * stride + (k == piece ? part_floats(pl) : 0);
            const float mk = __ldcg(w + (int64_t)rows * kLatent + r), lk = __ldcg(w + (int64_t)rows * (kLatent + 1) + r);
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(w + (int64_t)r * kLatent + ch));
            const float f = m == -INFINITY ? 1.f : ex2(mk - m);
            l += lk * f;
            acc = make_float4(acc.x + x.x * f, acc.y + x.y * f, acc.z + x.z * f, acc.w + x.w * f);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t out = (int64_t)(t.t0 + tok) * p.H + head, e = out * kLatent + ch;
        if (p.o_bf16)
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + e) =
                make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + e) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (ch == 0 && p.lse) p.lse[out] = l == 0.f ? -INFINITY : (log2f(l) + m) * kLn2;
    }
}

// ---------------------------------------------------------------------------
// host

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// How a call is split.  Tiles: all heads of as many tokens as 64 rows hold, or with more than 64 heads
// equal parts of one token's.
Plan plan_of(int64_t N, int64_t tokens, int H, int64_t max_tokens) {
    Plan pl;
    memset(&pl, 0, sizeof(pl));
    const int64_t avg = (tokens + N - 1) / N;  // rows of a sequence
    pl.parts = (H + kTileRows - 1) / kTileRows;
    pl.hp = (int)round_up((H + pl.parts - 1) / pl.parts, 8);
    pl.parts = (H + pl.hp - 1) / pl.hp;
    pl.tk = (int)std::max<int64_t>(1, std::min<int64_t>(kTileRows / pl.hp, avg));
    pl.n = (int)round_up(pl.hp * pl.tk, 16);
    const int64_t tiles = (avg + pl.tk - 1) / pl.tk * pl.parts;
    pl.G = tiles >= 4 ? 4 : tiles >= 2 ? 2 : 1;
    const int64_t sms = std::max(sm_count() / pl.G, 1);
    // (a sequence of nq rows has at most nq / (rows of a unit) + 1 units)
    const int64_t most_units = units_of(pl, tokens) + N, per = (max_tokens + kStep - 1) / kStep + kPad;
    pl.cut = 1;
    pl.pieces = (int)std::max<int64_t>(1, std::min(sms, (most_units * per + kMinPiece - 1) / kMinPiece));
    const int64_t q = (int64_t)pl.hp * pl.tk * kRow * 2, ps = (int64_t)pl.n * 128;
    const int64_t room = kMaxSmem - 1024 - (int64_t)round_up(sizeof(Bars), 128) - round_up(q, 1024) - round_up(ps, 1024);
    pl.shared = 2;
    pl.units = (int)std::min<int64_t>(kMaxUnits, (room - 2 * kSharedBytes) / kUnitBytes);
    pl.at_p = (uint32_t)round_up(q, 1024);
    pl.at_units = pl.at_p + (uint32_t)round_up(ps, 1024);
    pl.at_shared = pl.at_units + pl.units * kUnitBytes;
    pl.at_bars = pl.at_shared + pl.shared * kSharedBytes;
    return pl;
}

size_t plan_bytes(const Plan &pl) {
    return pl.cut ? (size_t)pl.pieces * pl.G * 2 * pl.hp * pl.tk * (kLatent + 2) * sizeof(float) : 0;
}

bool encode_tensors(const AttnLatentParams &p, const Plan &pl, CUtensorMap *mq, CUtensorMap *mc) {
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
    const cuuint64_t cd[2] = {(cuuint64_t)kRow, (cuuint64_t)p.c.n_pages * p.c.P};
    const cuuint64_t cs[1] = {(cuuint64_t)kRow * 2};
    const cuuint32_t cb[2] = {64, (cuuint32_t)std::min(p.c.P, kStep)};
    if (r == CUDA_SUCCESS)
        r = enc(mc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.c.rows, cd, cs, cb, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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
    CUtensorMap mq, mc;
    if (!encode_tensors(p, pl, &mq, &mc)) return KDA_ERR_CUDA;
    static DeviceOnce configured;
    const int dev = current_device();
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(attn_latent_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) {
            set_error("attn_latent: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    attn_latent_kernel<<<pl.pieces * pl.G, kThreads, kMaxSmem, st>>>(mq, mc, a);
    note_launch();
    kda_status s = check_launch("attn_latent_kernel");
    if (!pl.cut || s != KDA_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pl.pieces * pl.G, std::max(1, pl.hp * pl.tk / 8));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // starts while the first kernel ends; waits for it before it reads
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_latent_join_kernel, a);
    note_launch();
    if (e != cudaSuccess) {
        set_error("attn_latent_join_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return check_launch("attn_latent_join_kernel");
}

}  // namespace kda
