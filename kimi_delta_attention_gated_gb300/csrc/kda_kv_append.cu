// kda_kv_append.cu -- appends keys and values to a paged 8-bit cache, with the keys (and the
// step's queries) rotated on the way.
//
// The cache holds e4m3 codes [pages, Hk, P, D] and one scale for each (page, head).  Scales
// are powers of two, 2^e with the smallest e that keeps the block's values within 448:
//   - e4m3 is a floating type, so a finer scale would add no precision, only range;
//   - when a later token of a part-filled page is larger, the page's earlier codes move to
//     the new scale by an exact exponent shift (only codes that become subnormal are
//     rounded again), so the order in which tokens arrive hardly matters.
// A page whose first token is written here is taken as empty: its old scale is not read.
//
// The bound is memory.  The tokens of one call that fall into one page are a run; one CTA takes
// a run and some of the heads, holds the (rotated) values in registers between the pass that
// finds each head's largest value and the pass that writes codes, so everything is read
// once, and has the next heads' rows on their way meanwhile.  One token per sequence (a
// decode step) has a warp for each (sequence, head).  Queries are rotated by further CTAs
// of the same launch, or in a launch of their own beside the last runs.
// Eight prompts of [512, 16384] tokens, 32 query and 8 cache heads of 128, rotated keys written
// too: 300 us, 83 % of a copy's rate: the runs 117 us (instructions, 65 % of the issue slots, and a
// barrier for each head), the queries 183 us (88 %).  One token each of 256 sequences: 5.5 us;
// 37 pieces of [1, 100] tokens: 4.9 us, launch and latency.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kStepThreads = 256;  // of a decode step's CTA
constexpr int kRoom = 1024;  // cos / sin pairs of a query tile

struct Grid {
    int q_tile;     // tokens of a query CTA
    int n_kv;       // CTAs of the keys and values; the query CTAs follow
    int heads;      // heads of a run's CTA
    int head_parts; // CTAs that share a run's heads
};

// Tokens of sequence n in this call, clamped to the tensors.
__device__ __forceinline__ void new_tokens(const AppendParams &p, int n, int64_t &t0, int &len) {
    int64_t a = p.cu_seqlens[n], b = p.cu_seqlens[n + 1];
    a = max((int64_t)0, min(a, p.tokens));
    b = max(a, min(b, p.tokens));
    t0 = a;
    len = (int)(b - a);
}

// Pages that the new tokens of sequence n touch.
__device__ __forceinline__ int runs_of(const AppendParams &p, int n) {
    int64_t t0;
    int len;
    new_tokens(p, n, t0, len);
    const int ctx = max(p.c.lens[n], 0);
    return len > 0 ? (int)(((int64_t)ctx + len - 1) / p.c.P - ctx / p.c.P) + 1 : 0;
}

// Position of token t (-> its angle), by bisection of cu_seqlens.  Lengths and rows are int32, their
// sum is not: positions are unsigned.
__device__ __forceinline__ uint32_t position_of(const AppendParams &p, int64_t t) {
    if (!p.cu_seqlens) return max(p.c.lens[t], 0);
    int lo = 0, hi = p.c.N - 1;  // the last sequence that starts at or before t
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (p.cu_seqlens[m] <= t)
            lo = m;
        else
            hi = m - 1;
    }
    return (uint32_t)max(p.c.lens[lo], 0) + (uint32_t)(t - max(p.cu_seqlens[lo], 0));  // clamped as in new_tokens
}

// One query tile; rows of no sequence are left out.
template <int THREADS>
__device__ __forceinline__ void rotate_queries(const AppendParams &p, int tile, int q_tile, float2 *cs, uint32_t *pos) {
    int64_t t0 = (int64_t)tile * q_tile, t1 = min(t0 + q_tile, p.tokens);
    if (p.cu_seqlens) {
        t0 = max(t0, (int64_t)p.cu_seqlens[0]);
        t1 = min(t1, (int64_t)p.cu_seqlens[p.c.N]);
        if (t0 >= t1) return;
    }
    const int n = (int)(t1 - t0), tid = threadIdx.x;
    for (int t = tid; t < n; t += THREADS) pos[t] = position_of(p, t0 + t);
    __syncthreads();
    fill_cos_sin(cs, p.rot, n, [&](int t) { return pos[t]; }, tid, THREADS);
    __syncthreads();
    const int64_t row = (int64_t)p.Hq * p.c.D;
    rotate_rows<__nv_bfloat16>(p.q + t0 * p.q_stride, p.q_stride, p.q_out + t0 * row, row, cs, p.rot, n, p.Hq, p.c.D, tid,
                               THREADS);
}

// The scale's exponent of a block whose new values reach amax; off: tokens it already holds.
__device__ __forceinline__ int block_exp(float amax, int off, int old) {
    const int need = scale_exp(amax);
    return off > 0 ? max(need, old) : need;
}

// ---------------------------------------------------------------------------
// runs (any number of tokens per sequence)

// The queries of a long call, in a launch of their own: their CTAs need half the registers of
// a run's.
__global__ void __launch_bounds__(kStepThreads, 8) append_queries_kernel(const __grid_constant__ AppendParams p, int q_tile) {
    __shared__ __align__(16) float2 cs[kRoom];
    __shared__ uint32_t s_pos[kRoom];
    rotate_queries<kStepThreads>(p, blockIdx.x, q_tile, cs, s_pos);
    // Its CTAs start while the runs' last ones are at work, and share nothing with them; the launch
    // must not end before the runs' has.
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int P>
__global__ void __launch_bounds__(P *D / 16, 1024 / (P * D / 16)) append_run_kernel(const __grid_constant__ AppendParams p,
                                                                                   const __grid_constant__ Grid g) {
    constexpr int kThreads = P * D / 16, kWarps = kThreads / 32;
    extern __shared__ __align__(16) float2 cs[];
    __shared__ uint32_t s_pos[kRoom];
    __shared__ int s_seq, s_run;
    __shared__ int s_scan[kWarps];
    __shared__ float s_max[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the queries' launch, where there is one
    if ((int)blockIdx.x >= g.n_kv) {
        rotate_queries<kThreads>(p, blockIdx.x - g.n_kv, g.q_tile, cs, s_pos);
        return;
    }
    const int values = blockIdx.x & 1, part = (blockIdx.x >> 1) % g.head_parts, unit = (blockIdx.x >> 1) / g.head_parts;
    // the unit-th run over all sequences
    if (tid == 0) s_seq = -1;
    __syncthreads();
    int before = 0;
    for (int n0 = 0; n0 < p.c.N; n0 += kThreads) {
        const int n = n0 + tid;
        const int r = n < p.c.N ? runs_of(p, n) : 0;
        int x = r;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_scan[warp] = x;
        __syncthreads();
        int base = before, total = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += s_scan[w];
            total += s_scan[w];
        }
        const int first = base + x - r;
        if (r > 0 && unit >= first && unit < first + r) {
            s_seq = n;
            s_run = unit - first;
        }
        before += total;
        __syncthreads();
        if (before > unit) break;
    }
    const int seq = s_seq;
    if (seq < 0) return;
    int64_t t0;
    int len;
    new_tokens(p, seq, t0, len);
    const int ctx = max(p.c.lens[seq], 0), block = ctx / P + s_run;
    const int64_t pos0 = max((int64_t)block * P, (int64_t)ctx);
    const int off = (int)(pos0 - (int64_t)block * P);  // tokens the page holds already
    t0 += pos0 - ctx;
    const int n = min(P - off, len - (int)(pos0 - ctx));
    int page = block < p.c.max_blocks ? p.c.block_table[(int64_t)seq * p.c.max_blocks + block] : -1;
    if (page >= p.c.n_pages) page = -1;  // no such page: the tokens are dropped (their rotated copies are not)

    const int64_t stride = values ? p.v_stride : p.k_stride;
    const bool turned = !values && p.rot.R > 0;
    const int h0 = part * g.heads, h1 = min(h0 + g.heads, p.c.Hk), np = p.rot.R >> 1;
    // This thread's share of every head: two 16-byte pieces of one token, which in the rotated
    // part hold each other's partners and use the same eight cos / sin pairs.
    constexpr int U = D / 16;
    const int t = tid / U, u = tid % U, nrot = turned ? p.rot.R >> 4 : 0;
    const bool live = t < n, apart = u < nrot && !p.rot.interleaved;
    const int c0 = apart ? 8 * u : 16 * u, c1 = apart ? 8 * u + np : 16 * u + 8;
    const __nv_bfloat16 *src = (values ? p.v : p.k) + (t0 + t) * stride + h0 * D;
    __nv_bfloat16 *turned_to = !values && p.k_out ? p.k_out + ((t0 + t) * p.c.Hk + h0) * D : nullptr;
    const int64_t block0 = (int64_t)page * p.c.Hk;
    uint8_t *codes = (values ? p.c.v : p.c.k) + (block0 + h0) * (P * D);
    float *scales = (values ? p.c.v_scale : p.c.k_scale) + block0;
    // Two heads' rows are on their way while a third is worked on: with one, each head took a
    // memory latency.
    constexpr int AHEAD = 2;
    uint4 raw[AHEAD][2];
    int old_scale[AHEAD];
    auto fetch = [&](int h, uint4 (&w)[2], int &old) {
        if (live && h < h1) {
            w[0] = __ldg(reinterpret_cast<const uint4 *>(src + c0));
            w[1] = __ldg(reinterpret_cast<const uint4 *>(src + c1));
        }
        src += D;
        // a page that holds earlier tokens: its scale (no other CTA writes it)
        old = off > 0 && page >= 0 && h < h1 ? exp_of_scale(scales[h]) : kScaleExpLo;
    };
#pragma unroll
    for (int b = 0; b < AHEAD; ++b) fetch(h0 + b, raw[b], old_scale[b]);
    if (turned) {
        fill_cos_sin_run(cs, p.rot, n, pos0, tid, kThreads);
        __syncthreads();
    }
    const float2 *turns = cs + t * np;
    for (int hb = h0; hb < h1; hb += AHEAD)
#pragma unroll
    for (int b = 0; b < AHEAD; ++b) {
        const int h = hb + b;
        if (h >= h1) break;
        float y[2][8];
        float amax = 0.f;
        const int old = old_scale[b];
        if (live) {
            Vec16<__nv_bfloat16>::load(raw[b][0], y[0]);
            Vec16<__nv_bfloat16>::load(raw[b][1], y[1]);
            if (u < nrot) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const float4 w = cs_two(turns, 8 * u + i, np);
                    const float2 w0 = make_float2(w.x, w.y), w1 = make_float2(w.z, w.w);
                    if (p.rot.interleaved) {
                        float *z = &y[i >> 2][2 * (i & 3)];
                        turn_pair(z[0], z[1], w0, p.rot.magnitude, z[0], z[1]);
                        turn_pair(z[2], z[3], w1, p.rot.magnitude, z[2], z[3]);
                    } else {
                        turn_pair(y[0][i], y[1][i], w0, p.rot.magnitude, y[0][i], y[1][i]);
                        turn_pair(y[0][i + 1], y[1][i + 1], w1, p.rot.magnitude, y[0][i + 1], y[1][i + 1]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(fmaxf(amax, fabsf(y[0][i])), fabsf(y[1][i]));  // no NaN
            if (turned_to) {
                *reinterpret_cast<uint4 *>(turned_to + c0) = Vec16<__nv_bfloat16>::store(y[0]);
                *reinterpret_cast<uint4 *>(turned_to + c1) = Vec16<__nv_bfloat16>::store(y[1]);
            }
        }
        if (turned_to) turned_to += D;
        fetch(h + AHEAD, raw[b], old_scale[b]);
        if (page < 0) continue;
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
        if (lane == 0) s_max[h & 1][warp] = amax;
        __syncthreads();  // also: every thread has read this head's old scale
        auto largest = [&] { return __uint_as_float(__reduce_max_sync(0xffffffffu, lane < kWarps ? __float_as_uint(s_max[h & 1][lane]) : 0u)); };
        amax = largest();
        if (isinf(amax)) {  // rare: the largest finite value, and NaN in the infinities' places
            amax = 0.f;
            if (live) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    amax = fmaxf(amax, finite_abs(y[i >> 3][i & 7]));
                    y[i >> 3][i & 7] = no_infinity(y[i >> 3][i & 7]);
                }
            }
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            __syncthreads();
            if (lane == 0) s_max[h & 1][warp] = amax;
            __syncthreads();
            amax = largest();
        }
        const int e = block_exp(amax, off, old);
        if (off > 0 && e > old) {
            const float f = exp2_int(max(old - e, -126));
            uint32_t *w = reinterpret_cast<uint32_t *>(codes);
            for (int i = tid; i < off * D / 4; i += kThreads) w[i] = rescale_codes(w[i], f);
        }
        if (tid == 0) scales[h] = exp2_int(e);
        const float inv = exp2_int(-e);
        if (live) {
            auto put = [&](const float (&y)[8], int c) {
                uint2 w;
                w.x = e4m3x2(y[0] * inv, y[1] * inv) | e4m3x2(y[2] * inv, y[3] * inv) << 16;
                w.y = e4m3x2(y[4] * inv, y[5] * inv) | e4m3x2(y[6] * inv, y[7] * inv) << 16;
                *reinterpret_cast<uint2 *>(codes + (off + t) * D + c) = w;
            };
            put(y[0], c0);
            put(y[1], c1);
        }
        codes += P * D;
    }
}

// ---------------------------------------------------------------------------
// one token per sequence: a warp for each (sequence, head, keys or values)

template <int D>
__global__ void __launch_bounds__(kStepThreads) append_step_kernel(const __grid_constant__ AppendParams p,
                                                                   const __grid_constant__ Grid g) {
    constexpr int kThreads = kStepThreads, kWarps = kThreads / 32;
    constexpr int C = D / 32;  // channels of a lane
    __shared__ __align__(16) float2 cs[kRoom];
    __shared__ uint32_t s_pos[kRoom];
    if ((int)blockIdx.x >= g.n_kv) {
        rotate_queries<kThreads>(p, blockIdx.x - g.n_kv, g.q_tile, cs, s_pos);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (item >= (int64_t)p.c.N * p.c.Hk * 2) return;
    const int values = (int)(item & 1), h = (int)((item >> 1) % p.c.Hk), seq = (int)((item >> 1) / p.c.Hk);
    const __nv_bfloat16 *x = values ? p.v + seq * p.v_stride + h * D : p.k + seq * p.k_stride + h * D;
    const int c0 = lane * C, R = p.rot.R, half = R >> 1;
    // the token's row and the place it goes to do not depend on each other: both loads are in flight
    float own[C], other[C];
    const bool turned = !values && c0 < R;
    const bool second = turned && !p.rot.interleaved && c0 >= half;
    const int partner = !turned || p.rot.interleaved ? c0 : second ? c0 - half : c0 + half;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        own[i] = __bfloat162float(x[c0 + i]);
        other[i] = __bfloat162float(x[partner + i]);
    }
    const int ctx = max(p.c.lens[seq], 0), block = ctx / p.c.P, off = ctx - block * p.c.P;
    int page = block < p.c.max_blocks ? p.c.block_table[(int64_t)seq * p.c.max_blocks + block] : -1;
    if (page >= p.c.n_pages) page = -1;
    float y[C];
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = own[i];
    if (turned) {
        if (p.rot.interleaved) {
#pragma unroll
            for (int i = 0; i < C / 2; ++i) {
                float c, s;
                cos_sin_turn((uint64_t)(int64_t)ctx * turn_of(__ldg(p.rot.inv_freq + c0 / 2 + i)), c, s);
                turn_pair(own[2 * i], own[2 * i + 1], make_float2(c, s), p.rot.magnitude, y[2 * i], y[2 * i + 1]);
            }
        } else {
            const int j0 = second ? partner : c0;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float c, s;
                cos_sin_turn((uint64_t)(int64_t)ctx * turn_of(__ldg(p.rot.inv_freq + j0 + i)), c, s);
                y[i] = diff_of_products(own[i], c, second ? -other[i] : other[i], s) * p.rot.magnitude;
            }
        }
    }
    if (!values && p.k_out) {
#pragma unroll
        for (int i = 0; i < C; ++i) p.k_out[((int64_t)seq * p.c.Hk + h) * D + c0 + i] = __float2bfloat16_rn(y[i]);
    }
    if (page < 0) return;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        amax = fmaxf(amax, finite_abs(y[i]));
        y[i] = no_infinity(y[i]);
    }
    amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
    const int64_t blk = (int64_t)page * p.c.Hk + h;
    float *scales = values ? p.c.v_scale : p.c.k_scale;
    uint8_t *dst = (values ? p.c.v : p.c.k) + blk * p.c.P * D;
    const int old = exp_of_scale(scales[blk]), e = block_exp(amax, off, old);
    if (off > 0 && e > old) {
        const float f = exp2_int(max(old - e, -126));
        uint4 *w = reinterpret_cast<uint4 *>(dst);
        for (int i = lane; i < off * D / 16; i += 32) {
            uint4 u = w[i];
            u.x = rescale_codes(u.x, f);
            u.y = rescale_codes(u.y, f);
            u.z = rescale_codes(u.z, f);
            u.w = rescale_codes(u.w, f);
            w[i] = u;
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) scales[blk] = exp2_int(e);
    const float inv = exp2_int(-e);
#pragma unroll
    for (int i = 0; i < C; i += 2)
        *reinterpret_cast<uint16_t *>(dst + (int64_t)off * D + c0 + i) = (uint16_t)e4m3x2(y[i] * inv, y[i + 1] * inv);
}

template <int D, int P>
kda_status run(const AppendParams &p, Grid g, cudaStream_t st) {
    constexpr int THREADS = P * D / 16;
    // A sequence's n new tokens lie in at most n / P + 2 pages.
    const int64_t runs = p.tokens / p.c.P + 2 * (int64_t)p.c.N;
    g.q_tile = p.q ? rotary_tile_tokens(p.Hq, p.c.D, p.rot.R, 8, THREADS, kRoom) : 1;
    if (g.q_tile > kRoom) g.q_tile = kRoom;
    const int64_t q_ctas = p.q ? (p.tokens + g.q_tile - 1) / g.q_tile : 0;
    // A CTA takes all heads of its run, so that cos and sin are formed once, unless the GPU
    // would be left with fewer than four CTAs per SM.
    g.heads = p.c.Hk;
    while (g.heads > 1 && runs * 2 * ((p.c.Hk + g.heads - 1) / g.heads) < 4ll * sm_count()) g.heads = (g.heads + 1) / 2;
    g.head_parts = (p.c.Hk + g.heads - 1) / g.heads;
    const int64_t kv = runs * 2 * g.head_parts;
    if (kv + q_ctas > INT32_MAX) {
        set_error("kda_kv_append: too many tokens");
        return KDA_ERR_UNSUPPORTED;
    }
    g.n_kv = (int)kv;
    // Two launches where the queries alone fill the GPU, four CTAs an SM or more.  One launch and two,
    // 32/8 heads of 128, rotated keys kept: 1200 tokens 12.3 and 14.1 us, 2500 23.7 and 23.1, 5000 35.5
    // and 32.4, 9000 60 and 54, 20000 106 and 91, 60000 308 and 262; 16/2 heads of 64, pages of 16: 9000
    // tokens 14.8 and 14.4, 40000 51 and 46.
    const bool apart = q_ctas > 4ll * sm_count();
    size_t smem = (size_t)p.c.P * p.rot.R / 2 * sizeof(float2);
    if (p.q && !apart && smem < kRoom * sizeof(float2)) smem = kRoom * sizeof(float2);
    if (smem > 32 * 1024) {
        static DeviceOnce configured;
        const int dev = current_device();
        if (!configured.done(dev)) {
            if (cudaFuncSetAttribute(append_run_kernel<D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     64 * 1024) != cudaSuccess) {
                set_error("kv_append: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
                return KDA_ERR_CUDA;
            }
            configured.set(dev);
        }
    }
    append_run_kernel<D, P><<<(unsigned)(kv + (apart ? 0 : q_ctas)), THREADS, smem, st>>>(p, g);
    note_launch();
    if (apart) {
        const kda_status s = check_launch("append_run_kernel");
        if (s != KDA_OK) return s;
        int tile = rotary_tile_tokens(p.Hq, p.c.D, p.rot.R, 8, kStepThreads, kRoom);
        if (tile > kRoom) tile = kRoom;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((p.tokens + tile - 1) / tile));
        cfg.blockDim = dim3(kStepThreads);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, append_queries_kernel, p, tile);
        note_launch();
        if (e != cudaSuccess) {
            set_error("append_queries_kernel: %s", cudaGetErrorString(e));
            cudaGetLastError();
            return KDA_ERR_CUDA;
        }
        return check_launch("append_queries_kernel");
    }
    return check_launch("append_run_kernel");
}

}  // namespace

kda_status launch_kv_append(const AppendParams &p, cudaStream_t st) {
    if (p.tokens == 0) return KDA_OK;
    Grid g;
    if (!p.cu_seqlens) {
        constexpr int kWarps = kStepThreads / 32;
        g.q_tile = p.q ? rotary_tile_tokens(p.Hq, p.c.D, p.rot.R, 8, kStepThreads, kRoom) : 1;
        if (g.q_tile > kRoom) g.q_tile = kRoom;
        const int64_t q_ctas = p.q ? (p.tokens + g.q_tile - 1) / g.q_tile : 0;
        const int64_t kv = ((int64_t)p.c.N * p.c.Hk * 2 + kWarps - 1) / kWarps;
        g.n_kv = (int)kv;
        g.heads = g.head_parts = 1;
        const unsigned grid = (unsigned)(kv + q_ctas);
        if (p.c.D == 128)
            append_step_kernel<128><<<grid, kStepThreads, 0, st>>>(p, g);
        else
            append_step_kernel<64><<<grid, kStepThreads, 0, st>>>(p, g);
        note_launch();
        return check_launch("append_step_kernel");
    }
    if (p.c.D == 128) {
        if (p.c.P == 16) return run<128, 16>(p, g, st);
        if (p.c.P == 32) return run<128, 32>(p, g, st);
        if (p.c.P == 64) return run<128, 64>(p, g, st);
        return run<128, 128>(p, g, st);
    }
    if (p.c.P == 16) return run<64, 16>(p, g, st);
    if (p.c.P == 32) return run<64, 32>(p, g, st);
    if (p.c.P == 64) return run<64, 64>(p, g, st);
    return run<64, 128>(p, g, st);
}

}  // namespace kda
