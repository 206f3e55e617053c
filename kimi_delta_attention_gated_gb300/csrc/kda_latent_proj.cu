// kda_latent_proj.cu -- the products between the heads and the latent, with the projection W [H, 128
// key rows then 128 value rows, 512] as it is trained, no copy of it laid out:
//
//   queries  out[t, h] = [ sum_n q[t, h, n] W[h, n, :]  |  q[t, h, 128:192] turned by positions[t] ]
//   values   out[t, h] = sum_c o[t, h, c] W[h, 128 + ., c]
//   expand   k[t, h] = [ sum_c x[t, c] W[h, n, c], n < 128  |  x[t, 512:576] ],
//            v[t, h] = sum_c x[t, c] W[h, 128 + n, c]
//
// Matrix products of 128 tokens by NT outputs of one head on tcgen05, a tile a CTA, two
// CTAs on an SM (97 KB of shared memory each) so that one's copies and stores run beside the other's products.  W's inner index is the
// latent's channel: for the values and the expansion that is the sum's index (K-major), for the queries
// the output's (MN-major); the same bytes serve both.  Operands come by TMA, results leave by
// TMA through swizzled shared memory, which also cuts off the rows behind the last token.  The expansion of
// many tokens has a kernel of its own for pairs of SMs.
//
// What bounds it, and the floor by bytes or operations: queries, 256 tokens of 128 heads with turned channels 13.5 us (10), bytes
// of which half are W; 8192 of 32 heads 83 (61), each CTA's own chain of copy, product and output, two of which an SM
// holds.  Values, 256 tokens of 128 heads 12 (8.8); 8192 of 32 heads 58 (51), 88 % of a copy's rate.  Expansion, 100 tokens of 16 heads
// 4.6, a launch and the chain of one tile; 8192 of 32 heads 52 (36), see there.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "kda_chunk_common.cuh"
#include "kda_latent.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace {

using namespace tc;

constexpr int kTile = 128;  // tokens of a tile
constexpr int kThreads = 192, kMmaWarp = 4, kLoadWarp = 5, kTurnWarp = 6, kTurnWarps = 8;
constexpr uint32_t kBlock = kTile * 128;  // 64 channels of a tile's rows
constexpr uint32_t kSmSmem = 228 * 1024, kCtaSmem = 1024;  // an SM's shared memory; what a CTA takes beside its own
constexpr float kNaN = __builtin_nanf("");

__device__ int g_latent_product_timeouts = 0;

struct Bars {
    uint64_t full[4], empty[4], shared, done;
    uint32_t tmem;
    int abort;
};

// What: a LatentProduct.  The queries' sum has two K chunks of 64, which come in one go; the others'
// eight come through a ring.
template <int WHAT, int NT>
struct Cfg {
    static constexpr bool QUERIES = WHAT == kLatentQueries, EXPAND = WHAT == kLatentExpand;
    static constexpr int CHUNKS = QUERIES ? 2 : 8;
    static constexpr uint32_t A = kBlock, B = NT * 128;  // bytes of a chunk's operands
    static constexpr int STAGES = QUERIES ? 2 : NT == 256 ? 2 : NT == 128 ? 3 : 4;
    // the expansion's tile of shared channels: in the ring, as one more A chunk
    static constexpr uint32_t RING = STAGES * (A + B), SHARED = (CHUNKS % STAGES) * (A + B);
    static constexpr uint32_t BARS = RING;
    static constexpr int OUT_BLOCKS = NT / 64;
    static constexpr int NTILES = (QUERIES ? kLatent : EXPAND ? kHeadKey + kHeadValue : kHeadValue) / NT;  // of a head
    static constexpr uint32_t SMEM = BARS + sizeof(Bars) + 1024;
    static constexpr int THREADS = kThreads + (QUERIES ? 32 * kTurnWarps : 0);
    // where output block i is put together: the operands are through, the expansion's shared channels are not
    __host__ __device__ static constexpr uint32_t out_at(int i) { return EXPAND ? kBlock * (i + 1) : kBlock * i; }
    static_assert(!EXPAND || (kBlock * (OUT_BLOCKS + 1) <= RING && (SHARED == 0 || SHARED >= kBlock * (OUT_BLOCKS + 1))),
                  "the shared channels and the output lie apart");
    static_assert(kBlock * OUT_BLOCKS <= RING, "the output needs the operands' room");
    // The next launch may set up, and take its TMEM, while a CTA of this one still asks for its own.  It gets it, since
    // shared memory lets an SM hold two such CTAs, of either launch, whose columns fit together, and none beside a CTA
    // that takes all columns.  A third, or one of another kernel with less shared memory, could wait for a launch that
    // waits for it.
    static_assert(2 * NT <= 512 && 3 * (SMEM + kCtaSmem) > kSmSmem, "two CTAs an SM, and TMEM for both");
};

__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
__device__ __forceinline__ void tma_store_3d(const void *tmap, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(x), "r"(y), "r"(z), "r"(src)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *r) {
    uint32_t a[16], b[16];
    tmem_ld16(taddr, a);
    tmem_ld16(taddr + 16, b);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        asm volatile("" : "+r"(a[i]), "+r"(b[i]));  // uses stay behind the wait
        r[i] = __uint_as_float(a[i]);
        r[16 + i] = __uint_as_float(b[i]);
    }
}
// A barrier of the rows' warps that also says whether any of their threads has `x`.
__device__ __forceinline__ bool rows_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void rows_sync() { asm volatile("barrier.cta.sync 1, 128;" ::: "memory"); }

template <int WHAT, int NT>
__global__ void __launch_bounds__(Cfg<WHAT, NT>::THREADS)
    latent_product_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_out2,
                          const __grid_constant__ LatentProductParams p) {
    using F = Cfg<WHAT, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    Bars &b = *reinterpret_cast<Bars *>(sm + F::BARS);
    const int cta = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int NTILES = F::NTILES;
    const int nt = cta % NTILES, h = cta / NTILES % p.H, t0 = cta / NTILES / p.H * kTile;
    const bool with_shared = F::EXPAND && nt == 0;
    volatile int *abort_flag = &b.abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < F::STAGES; ++i) {
            mbar_init(b.full + i, 1);
            mbar_init(b.empty + i, 1);
        }
        mbar_init(&b.shared, 1);
        mbar_init(&b.done, 1);
        b.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&b.tmem, NT);
        tmem_relinquish();
    }
    next_may_start();
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    before_is_over();
    const uint32_t tb = b.tmem;
    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t polls) {
        for (uint32_t i = 0; i < polls; ++i) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*abort_flag) break;
        }
        *abort_flag = 1;
        return false;
    };
    if (warp == kLoadWarp) {
        if (elect_one()) {
            bool ok = true;
            int issued = 0;
            const int xh = F::EXPAND ? 0 : h;
            for (int i = 0; i < F::CHUNKS; ++i) {
                const int st = i % F::STAGES;
                if (i >= F::STAGES && !(ok = wait(b.empty + st, (i / F::STAGES - 1) & 1, kAttnPolls))) break;
                mbar_arrive_expect_tx(b.full + st, F::A + F::B);
                const uint32_t at = sb + st * (F::A + F::B);
                tma_load_3d(at, &map_x, b.full + st, i * 64, xh, t0);
                if (F::QUERIES)  // 64 of the sum's rows, the outputs in blocks of 64 channels
                    for (int x = 0; x < NT / 64; ++x)
                        tma_load_3d(at + F::A + x * 64 * 128, &map_w, b.full + st, nt * NT + x * 64, i * 64, h);
                else
                    tma_load_3d(at + F::A, &map_w, b.full + st, i * 64, (F::EXPAND ? 0 : kHeadKey) + nt * NT, h);
                ++issued;
            }
            if (with_shared && ok && (ok = wait(b.empty + F::CHUNKS % F::STAGES, (F::CHUNKS / F::STAGES - 1) & 1, kAttnPolls))) {
                mbar_arrive_expect_tx(&b.shared, kBlock);
                tma_load_3d(sb + F::SHARED, &map_x, &b.shared, kLatent, 0, t0);
            }
            // every copy lands before the CTA may end
            if (with_shared && ok) mbar_wait(&b.shared, 0, kAttnPolls);
            for (int i = issued > F::STAGES ? issued - F::STAGES : 0; i < issued; ++i)
                mbar_wait(b.full + i % F::STAGES, (i / F::STAGES) & 1, kAttnPolls);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        bool ok = true;
        const uint32_t id = idesc_bf16(kTile, NT, false, F::QUERIES);
        for (int i = 0; i < F::CHUNKS && ok; ++i) {
            const int st = i % F::STAGES;
            ok = __all_sync(0xffffffffu, wait(b.full + st, (i / F::STAGES) & 1, p.polls)) != 0;
            if (!ok) break;
            fence_after_sync();
            if (elect_one()) {
                const uint32_t at = sb + st * (F::A + F::B);
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mma_ss(tb, sdesc(at + x * 32, 16, 1024),
                           F::QUERIES ? sdesc(at + F::A + x * 2048, 64 * 128, 1024) : sdesc(at + F::A + x * 32, 16, 1024), id,
                           i > 0 || x > 0);
                mma_commit(b.empty + st);
            }
            __syncwarp();
        }
        if (elect_one()) {
            mma_commit(&b.done);
            mbar_wait(&b.done, 0, kAttnPolls);  // nothing may still run once the CTA has ended
        }
        __syncwarp();
    } else if (F::QUERIES && warp >= kTurnWarp) {
        // The shared channels of this CTA's part of the tile's rows, turned while the product runs, two channels a
        // lane, in warps of their own: 256 tokens, 128 heads 13.5 us (with four such warps 14.2, by the output's warps before
        // their output 17.2, and in a launch beside this one, the angles formed once for all heads, 14.8).
        constexpr int ROWS = kTile / NTILES / kTurnWarps;  // a warp's
        const int r0 = t0 + nt * (kTile / NTILES) + (warp - kTurnWarp) * ROWS, np = p.rot.R >> 1;
        const int at = np > 0 && lane < ROWS && r0 + lane < p.tokens ? __ldcg(p.positions + r0 + lane) : 0;
        uint32_t word[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (r0 + i < p.tokens)
                word[i] = __ldcg(reinterpret_cast<const uint32_t *>(p.x + (int64_t)(r0 + i) * p.x_stride + (int64_t)h * kHeadQuery + kHeadKey) + lane);
        const uint64_t turn = lane < np ? turn_of(__ldg(p.rot.inv_freq + lane)) : 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (np > 0) {
                float c, s;
                cos_sin_turn((uint64_t)(int64_t)__shfl_sync(0xffffffffu, at, i) * turn, c, s);
                word[i] = turn_word(word[i], c, s, p.rot);
            }
            if (r0 + i < p.tokens) reinterpret_cast<uint32_t *>(p.out + ((int64_t)(r0 + i) * p.H + h) * kRow + kLatent)[lane] = word[i];
        }
    } else {
        const int row = warp * 32 + lane;
        // the four warps go on or stop together, since they wait for each other at barriers
        bool ok = !rows_any(!wait(&b.done, 0, kAttnPolls) || *abort_flag);
        if (ok) {
            fence_after_sync();
            const uint32_t from = tb + ((uint32_t)(warp * 32) << 16);
#pragma unroll
            for (int i = 0; i < F::OUT_BLOCKS; ++i) {
                const uint32_t to = sb + F::out_at(i) + row * 128;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float x[32];
                    tmem_ld32(from + i * 64 + half * 32, x);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        st_shared_v4(to + (((half * 4 + q) ^ (row & 7)) << 4), pack_bf16x2(x[8 * q], x[8 * q + 1]),
                                     pack_bf16x2(x[8 * q + 2], x[8 * q + 3]), pack_bf16x2(x[8 * q + 4], x[8 * q + 5]),
                                     pack_bf16x2(x[8 * q + 6], x[8 * q + 7]));
                }
                fence_async_smem();
                rows_sync();
                if (threadIdx.x == 0) {
                    const int ch = nt * NT + i * 64;
                    if (F::EXPAND && ch >= kHeadKey)
                        tma_store_3d(&map_out2, sb + F::out_at(i), ch - kHeadKey, h, t0);
                    else
                        tma_store_3d(&map_out, sb + F::out_at(i), ch, h, t0);
                }
            }
            if (with_shared) {
                ok = !rows_any(!wait(&b.shared, 0, kAttnPolls));
                if (ok && threadIdx.x == 0) tma_store_3d(&map_out, sb + F::SHARED, kHeadKey, h, t0);
            }
            if (threadIdx.x == 0) {
                bulk_commit();
                bulk_wait_read_all();  // the shared memory is the CTA's until then
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tb, NT);
    if (*abort_flag) {  // a bounded wait gave up: the tile's outputs become NaN
        if (threadIdx.x == 0) bulk_wait_all();
        __syncthreads();
        const __nv_bfloat16 nan = __float2bfloat16_rn(kNaN);
        for (int r = threadIdx.x; r < kTile && t0 + r < p.tokens; r += F::THREADS) {
            const int64_t head = (int64_t)(t0 + r) * p.H + h;
            if (F::EXPAND) {
                for (int i = nt * NT; i < nt * NT + NT; ++i)
                    *(i < kHeadKey ? p.out + head * kHeadQuery + i : p.out2 + head * kHeadValue + i - kHeadKey) = nan;
                for (int i = kHeadKey; i < kHeadQuery && with_shared; ++i) p.out[head * kHeadQuery + i] = nan;
            } else {
                const int width = F::QUERIES ? kRow : kHeadValue;
                for (int i = 0; i < NT; ++i) p.out[head * width + nt * NT + i] = nan;
            }
        }
        if (threadIdx.x == 0) atomicAdd(&g_latent_product_timeouts, 1);
    }
}

// ---------------------------------------------------------------------------
// The expansion of many tokens, by pairs of CTAs: one product of 256 tokens by a head's 256 outputs on both SMs'
// tensor cores (cta_group::2), each CTA with its own 128 tokens and half of the head's rows of W.
// One CTA's tiles of 128 by 256 are bound by shared memory's 128 bytes a cycle: a step of 16 channels takes 12 KB out and
// 12 KB of copies in, 192 cycles for 128 of the tensor core.  Here W's 128 KB stay where they are for
// all tokens of a head, so that a step takes 8 KB out and 4 KB in.  A pair takes a run of (head,
// 256 tokens) in this order; the next head's W replaces the last's chunk by chunk; outputs leave while the
// next product runs, in the other half of TMEM.
// 8192 tokens, 32 heads: 52 us (tiles of 128 by 256: 68), 1.3 PFLOP/s.  A product takes 5600 cycles, of which the
// tensor core's rate would be 4096, and the stores of its outputs about as many beside it: without them it is 42 us, without
// the products 50: a warp's store covers 64 bytes of eight rows, and at 3.4 TB/s that is far below what the bytes need (28).

constexpr int kPairTokens = 256, kPairStages = 6, kChunks = kLatent / 64;
constexpr uint32_t kPairA = kChunks * kBlock, kPairBars = kPairA + kPairStages * kBlock;
constexpr uint32_t kSettlePolls = 256;  // a millisecond
constexpr int kPairThreads = 448, kPairMmaWarp = 8, kPairLoadWarp = 9, kPairSharedWarp = 10;

struct PairBars {
    uint64_t a_full[kPairStages], w_full[kChunks], acc_empty[2];   // the first CTA's, for both
    uint64_t a_empty[kPairStages], w_empty[kChunks], acc_full[2];  // each CTA's
    uint64_t drain, never;
    uint32_t tmem;
    int abort;
};
constexpr uint32_t kPairSmem = kPairBars + sizeof(PairBars) + 1024;
static_assert(kPairSmem <= 232448, "shared memory");
static_assert(kPairSmem + kCtaSmem + Cfg<kLatentValues, 64>::SMEM + kCtaSmem > kSmSmem, "an SM for itself: all of TMEM is its own");

__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// As tma_load_3d, the bytes counted on a barrier of either CTA.
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const void *tmap, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_load_5d(uint32_t dst, const void *tmap, uint32_t bar, int x, int v) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
        "%3, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(0), "r"(v), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives at `bar` of both CTAs when what this thread issued so far is through.
__device__ __forceinline__ void pair_commit(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// 16 lanes of 64 columns: of each 8 columns a thread has 2 (lane % 4) and the next, of row lane / 4 (registers 0, 1)
// and of the row eight further (2, 3).
__device__ __forceinline__ void tmem_ld_quads(uint32_t taddr, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
          "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
          "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ bool pair_try_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    latent_expand_pair_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                              const __grid_constant__ LatentProductParams p, int tiles) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    PairBars &b = *reinterpret_cast<PairBars *>(sm + kPairBars);
    const uint32_t rank = blockIdx.x & 1, lead = in_cta(sb + kPairBars, 0);  // the first CTA's barriers
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t items = (int64_t)tiles * p.H, pairs = gridDim.x >> 1, i0 = (blockIdx.x >> 1) * items / pairs,
                  i1 = ((blockIdx.x >> 1) + 1) * items / pairs;
    volatile int *abort_flag = &b.abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(b.a_full + i, 1);
            mbar_init(b.a_empty + i, 1);
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(b.w_full + i, 1);
            mbar_init(b.w_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b.acc_empty + i, 16);  // the rows' warps of both
            mbar_init(b.acc_full + i, 1);
        }
        mbar_init(&b.drain, 1);
        mbar_init(&b.never, 1);
        b.abort = 0;
        fence_mbar_init();
    }
    if (warp == kPairMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&b.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    next_may_start();
    fence_before_sync();
    __syncthreads();
    pair_sync();
    fence_after_sync();
    before_is_over();
    const uint32_t tb = b.tmem;
    auto give_up = [&] {  // both CTAs stop
        *abort_flag = 1;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(smem_u32(&b.abort), rank ^ 1)), "r"(1) : "memory");
        return false;
    };
    auto wait = [&](uint64_t *bar, uint32_t parity, uint32_t polls) {
        for (uint32_t i = 0; i < polls; ++i) {
            if (pair_try_wait(bar, parity)) return true;
            if (*abort_flag) return false;
        }
        return give_up();
    };
    if (warp == kPairLoadWarp) {
        if (elect_one()) {
            bool ok = true;
            uint32_t c = 0, heads = 0;  // chunks of tokens so far; heads
            for (int64_t i = i0; i < i1 && ok; ++i) {
                const int h = (int)(i / tiles), t = (int)(i - (int64_t)h * tiles);
                const bool fresh = i == i0 || t == 0;
                for (int k = 0; k < kChunks && ok; ++k, ++c) {
                    if (fresh) {
                        if (heads > 0) ok = wait(b.w_empty + k, (heads - 1) & 1, kAttnPolls);
                        if (!ok) break;
                        if (rank == 0) mbar_arrive_expect_tx(b.w_full + k, 2 * kBlock);
                        pair_load_5d(sb + k * kBlock, &map_w, lead + offsetof(PairBars, w_full) + k * 8, k * 64, 8 * h + 4 * rank);
                    }
                    const uint32_t st = c % kPairStages;
                    if (c >= kPairStages) ok = wait(b.a_empty + st, (c / kPairStages - 1) & 1, kAttnPolls);
                    if (!ok) break;
                    if (rank == 0) mbar_arrive_expect_tx(b.a_full + st, 2 * kBlock);
                    pair_load_3d(sb + kPairA + st * kBlock, &map_x, lead + offsetof(PairBars, a_full) + st * 8, k * 64, 0,
                                 t * kPairTokens + rank * kTile);
                }
                heads += fresh;
            }
            // What arrives here has to before the CTA may end: the products' signs for the last chunks, which come
            // behind the copies.  After a failure some never do: then the copies have a millisecond.
            for (uint32_t j = c > kPairStages ? c - kPairStages : 0; j < c && ok; ++j)
                ok = wait(b.a_empty + j % kPairStages, (j / kPairStages) & 1, kAttnPolls);
            for (int k = 0; k < kChunks && heads > 0 && ok; ++k) ok = wait(b.w_empty + k, (heads - 1) & 1, kAttnPolls);
        }
        __syncwarp();
    } else if (warp == kPairMmaWarp) {
        if (rank == 0 && elect_one()) {
            bool ok = true;
            const uint32_t id = idesc_bf16(kPairTokens, 256, false, false);
            uint32_t c = 0, heads = 0, n = 0;
            for (int64_t i = i0; i < i1 && ok; ++i, ++n) {
                const int t = (int)(i % tiles);
                const bool fresh = i == i0 || t == 0, last = i == i1 - 1 || t == tiles - 1;
                if (n >= 2) ok = wait(b.acc_empty + (n & 1), ((n >> 1) - 1) & 1, kAttnPolls);
                if (!ok) break;
                for (int k = 0; k < kChunks; ++k, ++c) {
                    const uint32_t st = c % kPairStages;
                    if (fresh) ok = wait(b.w_full + k, heads & 1, p.polls);
                    ok = ok && wait(b.a_full + st, (c / kPairStages) & 1, p.polls);
                    if (!ok) break;
                    fence_after_sync();
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        pair_mma(tb + (n & 1) * 256, sdesc(sb + kPairA + st * kBlock + x * 32, 16, 1024),
                                 sdesc(sb + k * kBlock + x * 32, 16, 1024), id, k > 0 || x > 0);
                    pair_commit(b.a_empty + st);
                    if (last) pair_commit(b.w_empty + k);
                }
                if (!ok) break;
                pair_commit(b.acc_full + (n & 1));
                heads += fresh;
            }
            asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&b.drain))
                         : "memory");
            mbar_wait(&b.drain, 0, kAttnPolls);  // nothing may still run once the CTAs have ended
        }
        __syncwarp();
    } else if (warp >= kPairSharedWarp) {
        // ---- the shared channels, a copy that depends on nothing else: 32 rows a warp, of 128 bytes, the next
        // tile's on their way while the last's are stored
        const int sub = (warp - kPairSharedWarp) * 32 + (lane >> 3), piece = lane & 7;
        uint4 r[8];
        auto load = [&](int64_t i) {
            const int64_t t0 = (i % tiles) * kPairTokens + rank * kTile + sub;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i < i1 && t0 + j * 4 < p.tokens)
                    r[j] = __ldcg(reinterpret_cast<const uint4 *>(p.x + (t0 + j * 4) * p.x_stride + kLatent) + piece);
        };
        load(i0);
        for (int64_t i = i0; i < i1; ++i) {
            const int64_t h = i / tiles, t0 = (i - h * tiles) * kPairTokens + rank * kTile + sub;
            uint4 y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = r[j];
            load(i + 1);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (t0 + j * 4 < p.tokens) reinterpret_cast<uint4 *>(p.out + ((t0 + j * 4) * p.H + h) * kHeadQuery + kHeadKey)[piece] = y[j];
        }
    } else {
        // ---- outputs: of the head's keys from the first four warps, of its values from the others, 64 bytes of a row
        // by four threads at once, from registers.  W's rows are taken in such an order (map_w) that a thread's
        // columns of 32 are eight outputs in a row: column 8 g + 2 c + e is output 8 c + 2 g + e.  (Through shared
        // memory and TMA they waited behind the copies of the next tokens, 2600 cycles for 16 KB, and their 32 KB are
        // two more places of the ring.)
        const int group = warp >> 2, r0 = (warp & 3) * 32;
        const int width = group == 0 ? kHeadQuery : kHeadValue;
        __nv_bfloat16 *out = (group == 0 ? p.out : p.out2) + (lane & 3) * 8;
        uint32_t n = 0;
        for (int64_t i = i0; i < i1; ++i, ++n) {
            const int h = (int)(i / tiles), t = (int)(i - (int64_t)h * tiles);
            const int64_t t0 = (int64_t)t * kPairTokens + rank * kTile + r0;
            if (!__all_sync(0xffffffffu, wait(b.acc_full + (n & 1), (n >> 1) & 1, kAttnPolls))) break;
            fence_after_sync();
            const uint32_t from = tb + ((uint32_t)r0 << 16) + (n & 1) * 256 + group * 128;
            // All is read before the first store, so that the product after the next never waits for those.
            uint4 y[4][4];  // 16 rows of 64 outputs each; in these a row's 32 outputs and the next, 8 rows further
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[32];
                tmem_ld_quads(from + ((uint32_t)(q >> 1) << 20) + (q & 1) * 64, x);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) asm volatile("" : "+f"(x[e]));  // uses stay behind the wait
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float *z = x + 16 * (e & 1) + 2 * (e >> 1);
                    y[q][e] = make_uint4(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[4], z[5]), pack_bf16x2(z[8], z[9]),
                                         pack_bf16x2(z[12], z[13]));
                }
            }
            fence_before_sync();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                                 lead + (uint32_t)offsetof(PairBars, acc_empty) + (n & 1) * 8)
                             : "memory");
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int64_t tok = t0 + e * 8 + (lane >> 2);
                __nv_bfloat16 *to = out + (tok * p.H + h) * width;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    if (tok < p.tokens) *reinterpret_cast<uint4 *>(to + 32 * v) = y[(e & 2) + (v >> 1)][(e & 1) * 2 + (v & 1)];
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) mbar_wait(&b.never, 0, kSettlePolls);
    pair_sync();
    fence_after_sync();
    if (warp == kPairMmaWarp) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tb) : "memory");
    if (*abort_flag) {  // a bounded wait gave up: this CTA's outputs become NaN
        __syncthreads();
        const __nv_bfloat16 nan = __float2bfloat16_rn(kNaN);
        for (int64_t i = i0; i < i1; ++i) {
            const int64_t h = i / tiles, t0 = (i - h * tiles) * kPairTokens + rank * kTile;
            for (int r = threadIdx.x; r < kTile && t0 + r < p.tokens; r += kPairThreads) {
                const int64_t head = (t0 + r) * p.H + h;
                for (int e = 0; e < kHeadQuery; ++e) p.out[head * kHeadQuery + e] = nan;
                for (int e = 0; e < kHeadValue; ++e) p.out2[head * kHeadValue + e] = nan;
            }
        }
        if (threadIdx.x == 0) atomicAdd(&g_latent_product_timeouts, 1);
    }
    pair_sync();  // the other's TMEM is given back
}

// ---------------------------------------------------------------------------
// host

// A tensor [rows, heads, dim] of bf16 in boxes of 64 channels x 1 head x box_rows.
bool encode(chunk::EncodeTiledFn enc, CUtensorMap *map, const void *base, int64_t dim, int64_t heads, int64_t rows,
            int64_t head_stride, int64_t row_stride, int box_heads, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)head_stride * 2, (cuuint64_t)row_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) set_error("latent product: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return r == CUDA_SUCCESS;
}

template <int WHAT, int NT>
kda_status run(const LatentProductParams &p, cudaStream_t st) {
    using F = Cfg<WHAT, NT>;
    chunk::EncodeTiledFn enc = reinterpret_cast<chunk::EncodeTiledFn>(tensor_map_encoder());
    if (!enc) {
        set_error("latent product: cuTensorMapEncodeTiled is not available from the driver");
        return KDA_ERR_CUDA;
    }
    CUtensorMap mx, mw, mo, mo2;  // (mo2: the expansion's values)
    if (!F::EXPAND) memset(&mo2, 0, sizeof(mo2));
    const int dim = F::QUERIES ? kHeadQuery : F::EXPAND ? kRow : kLatent, out = F::QUERIES ? kRow : F::EXPAND ? kHeadQuery : kHeadValue;
    const int heads = F::EXPAND ? 1 : p.H;
    // W as [heads, 256 rows, 512 channels]: 64 channels of 64 (queries) or NT rows of a head
    if (!encode(enc, &mx, p.x, dim, heads, p.tokens, dim, p.x_stride, 1, kTile) ||
        !encode(enc, &mw, p.w, kLatent, kHeadKey + kHeadValue, p.H, kLatent, (int64_t)(kHeadKey + kHeadValue) * kLatent,
                F::QUERIES ? 64 : NT, 1) ||
        !encode(enc, &mo, p.out, out, p.H, p.tokens, out, (int64_t)p.H * out, 1, kTile) ||
        (F::EXPAND && !encode(enc, &mo2, p.out2, kHeadValue, p.H, p.tokens, kHeadValue, (int64_t)p.H * kHeadValue, 1, kTile)))
        return KDA_ERR_CUDA;
    static DeviceOnce configured;
    const int dev = current_device();
    const auto kernel = latent_product_kernel<WHAT, NT>;
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM) != cudaSuccess) {
            set_error("latent product: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    const int64_t ctas = (p.tokens + kTile - 1) / kTile * p.H * F::NTILES;
    if (ctas > INT32_MAX || p.tokens > (1 << 30)) {
        set_error("latent product: too many tokens");
        return KDA_ERR_UNSUPPORTED;
    }
    const cudaError_t e = launch_beside_end(kernel, (unsigned)ctas, F::THREADS, F::SMEM, st, mx, mw, mo, mo2, p);
    return launched(e, "latent_product_kernel");
}

kda_status run_pairs(const LatentProductParams &p, cudaStream_t st) {
    chunk::EncodeTiledFn enc = reinterpret_cast<chunk::EncodeTiledFn>(tensor_map_encoder());
    if (!enc) {
        set_error("latent product: cuTensorMapEncodeTiled is not available from the driver");
        return KDA_ERR_CUDA;
    }
    CUtensorMap mx, mw;
    // W as [blocks of 32 rows][4][4][2][512 channels], the fours' order turned: see the kernel's outputs
    const cuuint64_t dims[5] = {(cuuint64_t)kLatent, 2, 4, 4, (cuuint64_t)p.H * 8};
    const cuuint64_t strides[4] = {kLatent * 2, 8 * kLatent * 2, 2 * kLatent * 2, 32 * kLatent * 2};
    const cuuint32_t box[5] = {64, 2, 4, 4, 4}, es[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(&mw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<__nv_bfloat16 *>(p.w), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        set_error("latent product: cuTensorMapEncodeTiled failed (%d)", (int)r);
        return KDA_ERR_CUDA;
    }
    if (!encode(enc, &mx, p.x, kRow, 1, p.tokens, kRow, p.x_stride, 1, kTile))
        return KDA_ERR_CUDA;
    static DeviceOnce configured;
    const int dev = current_device();
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(latent_expand_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem) != cudaSuccess) {
            set_error("latent product: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    const int64_t tiles = (p.tokens + kPairTokens - 1) / kPairTokens, pairs = std::min<int64_t>(sm_count() / 2, tiles * p.H);
    const cudaError_t e = launch_beside_end(latent_expand_pair_kernel, (unsigned)(2 * pairs), kPairThreads, kPairSmem, st, mx, mw, p, (int)tiles);
    return launched(e, "latent_expand_pair_kernel");
}

}  // namespace

int take_latent_product_timeouts(cudaStream_t st) {
    int n = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&n, g_latent_product_timeouts, sizeof(int), 0, cudaMemcpyDeviceToHost, st) !=
            cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_latent_product_timeouts, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) !=
            cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        set_error("latent product: cannot read the timeout counter: %s", cudaGetErrorString(cudaGetLastError()));
        return -1;
    }
    return n;
}

kda_status launch_latent_product(const LatentProductParams &p, cudaStream_t st) {
    if (p.tokens == 0) return KDA_OK;
    // Narrow tiles where wide ones would leave SMs without one.  Expansion by 64, 128 and 256 outputs: 100 tokens, 16
    // heads 5.4, 5.6, 7.6 us, 64 heads 7.5, 6.2, 7.9; 256 tokens, 72 heads 10.4, 7.7, 9.8, 128 heads 20.1, 15.6, 14.2.  By
    // tiles of 256 and by pairs, with 1.5 products of 256 tokens a pair 13.5, 13.5, with 1.7 11.5, 12.6, with 2.1 16.5, 14.9,
    // with 6.7 39.5, 29.2, with 13.5 (8192 tokens, 32 heads) 68.3, 52.1.  Values
    // by 64 and 128: 8 tokens, 32 heads 5.0, 5.3; 256 tokens, 72 heads 6.6, 7.5, 80 heads 10.5, 8.8.  The queries' short sum
    // gains nothing from them: by 64, 128 and 256, 8 tokens, 32 heads 5.1, 4.6, 4.4; 256 tokens, 128 heads 17.0, 14.9, 13.6.
    const int64_t wide = (p.tokens + kTile - 1) / kTile * p.H;
    if (p.what == kLatentQueries) return run<kLatentQueries, 256>(p, st);
    if (p.what == kLatentExpand)
        return wide * 4 < sm_count() ? run<kLatentExpand, 64>(p, st)
               : wide < sm_count()   ? run<kLatentExpand, 128>(p, st)
               : (p.tokens + kPairTokens - 1) / kPairTokens * p.H >= sm_count() && p.tokens < (1 << 30) ? run_pairs(p, st)
                                     : run<kLatentExpand, 256>(p, st);
    return wide < sm_count() ? run<kLatentValues, 64>(p, st) : run<kLatentValues, 128>(p, st);
}

}  // namespace kda
