// kda_latent_proj.cu -- the products between the heads and the latent, with the projection W [H, 128
// key rows then 128 value rows, 512] as it is trained, no copy of it laid out:
//
//   queries  out[t, h] = [ sum_n q[t, h, n] W[h, n, :]  |  q[t, h, 128:192] turned by positions[t] ]
//   values   out[t, h] = sum_c o[t, h, c] W[h, 128 + ., c]
//   expand   k[t, h] = [ sum_c x[t, c] W[h, n, c], n < 128  |  x[t, 512:576] ],
//            v[t, h] = sum_c x[t, c] W[h, 128 + n, c]
//
// Matrix products of 128 tokens by NT outputs of one head on tcgen05, a tile a CTA, two to three
// CTAs on an SM so that one's copies and stores run beside another's products.  W's inner index is the
// latent's channel: for the values and the expansion that is the sum's index (K-major), for the queries
// the output's (MN-major); the same bytes serve both.  Operands come by TMA, results leave by
// TMA through swizzled shared memory, which also cuts off the rows behind the last token.
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
constexpr int kThreads = 192, kMmaWarp = 4, kLoadWarp = 5;
constexpr uint32_t kBlock = kTile * 128;  // 64 channels of a tile's rows
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
    // where output block i is put together: the operands are through, the expansion's shared channels are not
    __host__ __device__ static constexpr uint32_t out_at(int i) { return EXPAND ? kBlock * (i + 1) : kBlock * i; }
    static_assert(!EXPAND || (kBlock * (OUT_BLOCKS + 1) <= RING && (SHARED == 0 || SHARED >= kBlock * (OUT_BLOCKS + 1))),
                  "the shared channels and the output lie apart");
    static_assert(kBlock * OUT_BLOCKS <= RING, "the output needs the operands' room");
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

// The queries' other channels, turned: a CTA's tokens have their angles formed once for all heads.  (In the
// products' CTAs, where each head's formed them anew, this was a quarter of the time.)
constexpr int kTurnTokens = 32;
template <int THREADS>
__device__ __forceinline__ void turn_shared(const LatentProductParams &p, int tile, int tokens, float2 *cs) {  // [tokens][R / 2]
    const int64_t t0 = (int64_t)tile * tokens;
    const int n = (int)min((int64_t)tokens, p.tokens - t0), np = p.rot.R >> 1, units = rotary_units(kShared, p.rot.R, p.rot.interleaved, 8);
    if (np > 0) {
        fill_cos_sin(cs, p.rot, n, [&](int t) { return __ldg(p.positions + t0 + t); }, threadIdx.x, THREADS);
        __syncthreads();
    }
    for (int i = threadIdx.x; i < n * p.H * units; i += THREADS) {
        const int row = i / units, u = i - row * units, t = row / p.H, h = row - t * p.H;
        rotate_unit<__nv_bfloat16>(p.x + (t0 + t) * p.x_stride + (int64_t)h * kHeadQuery + kHeadKey,
                                   p.out + ((t0 + t) * p.H + h) * kRow + kLatent, cs + t * np, u, p.rot.R, p.rot.interleaved,
                                   p.rot.magnitude);
    }
}
// In a launch of its own that runs beside the products': among their CTAs in one launch the turning ones
// would hold places that the products want (256 tokens, 128 heads: 27 and 15 us).  Where all fit the GPU at once
// it is one launch, which costs less on the host.
constexpr int kTurnThreads = 256;
__global__ void __launch_bounds__(kTurnThreads) latent_turn_kernel(const __grid_constant__ LatentProductParams p, int tokens) {
    __shared__ __align__(16) float2 cs[kTurnTokens * kShared / 2];
    turn_shared<kTurnThreads>(p, blockIdx.x, tokens, cs);
    // It shares nothing with the products' launch, but must not end before that has.
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int WHAT, int NT>
__global__ void __launch_bounds__(kThreads)
    latent_product_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                          const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_out2,
                          const __grid_constant__ LatentProductParams p, int turn_from, int turn_tokens) {
    using F = Cfg<WHAT, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(sm);
    if (F::QUERIES) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        if ((int)blockIdx.x >= turn_from) {
            turn_shared<kThreads>(p, blockIdx.x - turn_from, turn_tokens, reinterpret_cast<float2 *>(sm));
            return;
        }
    }
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
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
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
        for (int r = threadIdx.x; r < kTile && t0 + r < p.tokens; r += kThreads) {
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
    // turning CTAs with about four units a thread
    const int tokens = (int)std::max<int64_t>(1, std::min<int64_t>(kTurnTokens, 4 * kTurnThreads / (8 * p.H)));
    const int64_t turn_ctas = F::QUERIES ? (p.tokens + tokens - 1) / tokens : 0;
    const bool together = ctas + turn_ctas <= sm_count();
    kernel<<<(unsigned)(ctas + (together ? turn_ctas : 0)), kThreads, F::SMEM, st>>>(mx, mw, mo, mo2, p, (int)ctas, tokens);
    note_launch();
    const kda_status s = check_launch("latent_product_kernel");
    if (!F::QUERIES || together || s != KDA_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)turn_ctas);
    cfg.blockDim = dim3(kTurnThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, latent_turn_kernel, p, tokens);
    note_launch();
    if (e != cudaSuccess) {
        set_error("latent_turn_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return check_launch("latent_turn_kernel");
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
    // heads 5.4, 5.6, 7.6 us, 64 heads 7.5, 6.2, 7.9; 256 tokens, 72 heads 10.4, 7.7, 9.8, 128 heads 20.1, 15.6, 14.2.  Values
    // by 64 and 128: 8 tokens, 32 heads 5.0, 5.3; 256 tokens, 72 heads 6.6, 7.5, 80 heads 10.5, 8.8.  The queries' short sum
    // gains nothing from them: by 64, 128 and 256, 8 tokens, 32 heads 5.1, 4.6, 4.4; 256 tokens, 128 heads 17.0, 14.9, 13.6.
    const int64_t wide = (p.tokens + kTile - 1) / kTile * p.H;
    if (p.what == kLatentQueries) return run<kLatentQueries, 256>(p, st);
    if (p.what == kLatentExpand)
        return wide * 4 < sm_count() ? run<kLatentExpand, 64>(p, st)
               : wide < sm_count()   ? run<kLatentExpand, 128>(p, st)
                                     : run<kLatentExpand, 256>(p, st);
    return wide < sm_count() ? run<kLatentValues, 64>(p, st) : run<kLatentValues, 128>(p, st);
}

}  // namespace kda
