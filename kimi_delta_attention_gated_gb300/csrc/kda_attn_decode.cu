// kda_attn_decode.cu -- one query token per sequence against a paged 8-bit cache.
//
//   s_j = scale * q . (ks_j k_j),  o = sum_j e^(s_j - m) vs_j v_j / sum_j e^(s_j - m)
//
// with e4m3 codes k_j, v_j and one scale ks, vs for each (page, head).  Bound by the
// cache's bytes: each code is read once, for all query heads of its group.
//
// Products.  e4m3 fits f16 exactly, so codes are widened two at a time and multiplied with
// mma.sync in the transposed form: S^T = K q^T and O^T = V^T P^T, where the 16-row operand
// is the cache (16 tokens, then 16 value channels) and the 8-column one the query heads, so
// a group of up to 8 heads costs one product (16 heads: two).  tcgen05's 128-row tiles
// would leave 15 of 16 rows idle here, and the tensor work is far from the bound.
// Both operands' inner index may be permuted freely as long as both sides agree, so each
// lane takes 16 contiguous bytes of a row and no transposition through shared memory is
// needed; P goes from the one product's layout to the other's by movmatrix.
//
// The value scale is folded into P: with M the largest s_j + log2 vs_j so far less kRef,
// e_j = 2^(s_j - M) is summed for the denominator and e_j * vs_j * 2^(kTop - kRef), at most 2^15, is rounded to f16
// for the product, so pages of very different scales share one accumulator.  f16 takes up to
// 2^-25 from a weight below 2^-14.  That is nothing beside sums that hold a weight of 2^kTop, unless
// its value is near zero (a first token that takes nearly all the weight may have such a value):
// the output is then what the others make of it.  So a warp whose sums come out that small
// goes through its steps again (again_with_rest).
//
// Work split.  All (sequence, head, 32 tokens) steps are numbered in one line, kPad places
// before each head standing for what a head costs beside its steps, and the line is cut into
// equal pieces, one per CTA, whatever the lengths of the sequences are; every CTA finds its
// piece from the lengths on the device.  A head that one CTA covers is written at once, the
// others go through a workspace and attn_decode_join_kernel, which adds a head's pieces in
// their order, so results do not depend on timing.  Short sequences are not cut (decode_ctas).
//
// Copies.  Each warp has a ring of steps in shared memory, filled by TMA ahead of their use
// and across the borders of heads, without a barrier between warps.  The swizzle of the rows
// and the choice of the pieces a lane takes leave no bank conflict (64-channel values: two
// ways).  With 16-byte copies by each lane (cp.async) the load and store pipe was the bound,
// 148 us for 256 sequences of about 1000 tokens against 116 at that stage.
//
// 256 sequences of about 1000 tokens, 64 heads over 8 of 128, pages of 64: 97 us, 5.5 TB/s (81 % of
// a copy's rate); 8 of [8192, 131072] tokens, 40 heads over 8, pages of 16: 113 us, 6.0 TB/s (88 %);
// one of 1000 tokens: 9.0 us, both launches and their latencies.  The stream itself runs at
// 6.0 to 6.3 TB/s; the rest is about 8 us of finding the pieces, first copies, and joining.  128 heads
// over 8 (groups of 16), the same 256 sequences: 134 us; 255 registers leave an SM eight warps, and
// a step's chain of products, exponentials and products is the bound (issue slots 37 %, DRAM 53 %).
// 64 channels, 64 and 128 heads over 8: 69 and 87 us.
#include <cuda.h>
#include <cuda_fp16.h>

#include "kda_attn.cuh"
#include "kda_chunk_common.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kJoinMost = 512;   // threads of a joining CTA at most
constexpr int kStep = 32;       // tokens of a step
constexpr int kPad = 6;         // a head's own cost in steps
constexpr int kMinPiece = 8;   // places of a CTA at least
constexpr float kSlack = 2.f;   // the maximum in use may lie this far below the true one (log2)
constexpr int kTop = 12;        // a weight at that maximum is 2^kTop, times the scale's fraction below 2
// How far M lies below the maximum, and what the value scales are multiplied with to make up for it.  Sums of
// 2^(s - M) then stay within fp32 for value scales from 2^-126 to 2^120: M goes by a scale of at least
// 2^kLeastScale, so that each is at most 2^(kSlack + kRef - kLeastScale) = 2^92 (2^31 of them 2^123),
// and at least 2^(kRef - 120) where the scale decides, 2^24 above what is flushed.
constexpr int kRef = 18, kLeastScale = -72;
constexpr int kUp = 40;         // 2^-25 times 2^kUp is 2^15, and down to 2^-54 it stays normal in f16
constexpr float kLeast = 6.103515625e-5f;  // 2^-14, the least normal f16 number
constexpr float kNegInf = -INFINITY;

__device__ int g_attn_decode_timeouts = 0;

// Named barriers of some of a CTA's warps.
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void bar_arrive(int id, int threads) {
    asm volatile("barrier.cta.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <int D, int NT>
struct Cfg {
    static constexpr int ROWS = 8 * NT;                 // query heads of a unit
    static constexpr int KJ = D / 64;                   // 64-byte pieces of a key row
    static constexpr int VB = D / 8;                    // bytes of a value row per lane
    static constexpr int MT = D / 16;                   // 16-channel tiles of the output
    static constexpr int DEPTH = D == 128 ? 2 : 4;      // steps of a warp in flight
    static constexpr int HALF = 16 * D;                 // bytes of 16 rows
    static constexpr int KBYTES = kStep * D;            // a step's keys, then as many of values
    static constexpr int SLOT = 2 * KBYTES;
    static constexpr int PITCH = D + 4;                 // fp32 row of the merge buffer
    static constexpr int RING = kWarps * DEPTH * SLOT;
    static constexpr int SCALES = RING;                 // [warp][slot] {k, v of rows 0-15; of 16-31}
    static constexpr int BARS = SCALES + kWarps * DEPTH * 16;
    static constexpr int MERGE = BARS + kWarps * DEPTH * 8;
    static constexpr int SMEM = MERGE + 2 * ROWS * (PITCH + 2) * 4 + 1024;  // the ring starts on 1024 bytes
    static constexpr int CTAS = D == 128 && NT == 2 ? 2 : 3;  // per SM, by shared memory
    static constexpr int PART = ROWS * (D + 2);         // floats of one piece in the workspace
};

__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The four e4m3 codes of w as two pairs of f16.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The lesser of two pairs of f16 numbers, each by itself (of a NaN and a number the number).
__device__ __forceinline__ uint32_t min_half2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Adds the product of 16 tokens' weights, packed to f16 in the layout of the scores, with their
// values at v (v_at: this lane's pieces; live: tokens there are); REST: the weights are 2^kUp times
// what they stand for.
template <int D, int NT, bool REST>
__device__ __forceinline__ void add_products(float (&acc)[NT][D / 16][4], const uint32_t (&w)[NT][2], const uint8_t *v, int v_at0,
                                             int v_at1, int live) {
    using F = Cfg<D, NT>;
    const int t = threadIdx.x & 3;
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) pb[nt][e] = transpose8(w[nt][e]);
    uint32_t vw[4][F::VB / 4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint8_t *at = v + ((i & 1) ? v_at1 : v_at0) + (i >> 1) * (F::HALF / 2);
        if (F::VB == 16) {
            const uint4 x = *reinterpret_cast<const uint4 *>(at);
            vw[i][0] = x.x;
            vw[i][1] = x.y;
            vw[i][F::VB / 4 - 2] = x.z;
            vw[i][F::VB / 4 - 1] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(at);
            vw[i][0] = x.x;
            vw[i][1] = x.y;
        }
    }
    if (live < 16) {  // a zero weight would turn a NaN behind the last token into one
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (2 * t + (i & 1) + (i >> 1) * 8 >= live) {
#pragma unroll
                for (int x = 0; x < F::VB / 4; ++x) vw[i][x] = 0;
            }
    }
#pragma unroll
    for (int i = 0; i < F::VB / 4; ++i) {
        const uint32_t x = __byte_perm(vw[0][i], vw[1][i], 0x5140), y = __byte_perm(vw[0][i], vw[1][i], 0x7362);
        const uint32_t z = __byte_perm(vw[2][i], vw[3][i], 0x5140), u = __byte_perm(vw[2][i], vw[3][i], 0x7362);
        uint32_t x0, x1, y0, y1, z0, z1, u0, u1;
        widen(x, x0, x1);
        widen(y, y0, y1);
        widen(z, z0, z1);
        widen(u, u0, u1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (!REST) {
                mma_f16(acc[nt][2 * i], x0, x1, z0, z1, pb[nt][0], pb[nt][1]);
                mma_f16(acc[nt][2 * i + 1], y0, y1, u0, u1, pb[nt][0], pb[nt][1]);
                continue;
            }
            float a[4] = {}, b[4] = {};
            mma_f16(a, x0, x1, z0, z1, pb[nt][0], pb[nt][1]);
            mma_f16(b, y0, y1, u0, u1, pb[nt][0], pb[nt][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[nt][2 * i][e] = fmaf(a[e], exp2_int(-kUp), acc[nt][2 * i][e]);
                acc[nt][2 * i + 1][e] = fmaf(b[e], exp2_int(-kUp), acc[nt][2 * i + 1][e]);
            }
        }
    }
}

// A warp's sums over its steps s0, s0 + kWarps, .. of a unit anew, from global memory: the rows' M
// are known, and what f16 takes from a weight below 2^-14 is multiplied too, 2^kUp times as large.
// Seldom taken, and slow; a check in each step, with the rest at once, cost every call 5 to 15 %
// with groups above 8, and a look at the weights' least alone 5 %.
template <int D, int NT>
struct Again {
    uint32_t q[NT][D / 16][2];
    float row_scale[NT][2], M[NT][2], acc[NT][D / 16][4];
};
template <int D, int NT>
__device__ __noinline__ void again_with_rest(const DecodeParams &p, int n, int head, int len, int s0, int s1, Again<D, NT> &a) {
    using F = Cfg<D, NT>;
    const PagedCache &c = p.c;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[NT][F::MT][4] = {};
    for (int h = 2 * s0; h < 2 * s1; h += h & 1 ? 2 * kWarps - 1 : 1) {  // halves of steps
        const int live = len - 16 * h;
        if (live <= 0) break;
        const int page = __ldg(c.block_table + (int64_t)n * c.max_blocks + (16 * h >> c.p_shift));
        const bool good = (uint32_t)page < (uint32_t)c.n_pages;
        const int64_t block = (int64_t)(good ? page : 0) * c.Hk + head, at = ((block << c.p_shift) + (16 * h & (c.P - 1))) * D;
        const float ks = good ? c.k_scale[block] : __int_as_float(0x7fc00000),
                    vs = c.v_scale[block] * exp2_int(kTop - kRef);
        const uint8_t *v = c.v + at;
        const int v0 = 2 * t * D + g * F::VB;
        uint32_t codes = 0;  // values that are all zero (a cache not filled yet) add nothing
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < F::VB; x += 4)
                codes |= *reinterpret_cast<const uint32_t *>(v + v0 + (i & 1) * D + (i >> 1) * 8 * D + x);
        if (good && vs == vs && !__any_sync(0xffffffffu, codes & 0x7F7F7F7Fu)) continue;
        float S[NT][4] = {};
#pragma unroll
        for (int j = 0; j < F::KJ; ++j) {
            const uint8_t *k = c.k + at + g * D + 16 * (F::KJ * t + j);
            const uint4 x = *reinterpret_cast<const uint4 *>(k), y = *reinterpret_cast<const uint4 *>(k + 8 * D);
            const uint32_t wa[4] = {x.x, x.y, x.z, x.w}, wb[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a0, a1, a2, a3;
                widen(wa[i], a0, a2);
                widen(wb[i], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(S[nt], a0, a1, a2, a3, a.q[nt][4 * j + i][0], a.q[nt][4 * j + i][1]);
            }
        }
        uint32_t x[NT][2], r[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float w[4], z[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float m = a.M[nt][e & 1];
                w[e] = g + (e >> 1) * 8 < live ? ex2(S[nt][e] * (a.row_scale[nt][e & 1] * ks) - (m == kNegInf ? 0.f : m)) * vs : 0.f;
                z[e] = w[e] < kLeast ? (w[e] - __half2float(__float2half_rn(w[e]))) * exp2_int(kUp) : 0.f;
            }
            x[nt][0] = pack_half(w[0], w[1]);
            x[nt][1] = pack_half(w[2], w[3]);
            r[nt][0] = pack_half(z[0], z[1]);
            r[nt][1] = pack_half(z[2], z[3]);
        }
        add_products<D, NT, false>(acc, x, v, v0, v0 + D, live);
        add_products<D, NT, true>(acc, r, v, v0, v0 + D, live);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < F::MT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.acc[nt][j][e] = acc[nt][j][e];
}

// The factor that brings sums from one reference to another, as its square root: value scales far apart
// put references more than 126 powers of two apart, while the sums' sizes make up for it.
__device__ __forceinline__ float root_factor(float from, float to) { return to == kNegInf ? 1.f : ex2(0.5f * (from - to)); }
__device__ __forceinline__ float bring(float x, float root) { return x * root * root; }

// Tokens and steps of sequence n, its length clamped to what its block table can hold.
__device__ __forceinline__ int tokens_of(const PagedCache &c, int n) {
    const int64_t room = (int64_t)c.max_blocks * c.P;
    return (int)max((int64_t)0, min((int64_t)c.lens[n], min(room, (int64_t)INT32_MAX - kStep)));
}
__device__ __forceinline__ int steps_of(const PagedCache &c, int n) { return (tokens_of(c, n) + kStep - 1) / kStep; }

// Places of one unit (head, part of its group) of a sequence on the line.
__device__ __forceinline__ int places_of(int steps) { return steps ? steps + kPad : 0; }

// The line: sequence n's U units lie one after another, each places_of(steps) long, behind
// those of the sequences before.
struct Line {
    int64_t total;    // places of all sequences, one unit each
    int64_t mine;     // those before this thread's first sequence
    int first, last;  // this thread's sequences [first, last)
};
__device__ __forceinline__ Line measure_line(const PagedCache &c, int64_t *scan, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (c.N + threads - 1) / threads;
    Line l;
    l.first = min(tid * per, c.N);
    l.last = min(l.first + per, c.N);
    int64_t own = 0;
    for (int n = l.first; n < l.last; ++n) own += places_of(steps_of(c, n));
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
__device__ __forceinline__ int64_t piece_places(int64_t line, int ctas) {
    const int64_t s = (line + ctas - 1) / ctas;
    return s < kMinPiece ? kMinPiece : s;
}

// A run of places within one unit, and its steps [s0, s1) (none where it lies in the padding).
struct Segment {
    int n, u, steps, len;
    int s0, s1;
    int head;    // key/value head of unit u
    int places;  // of the line
};
__device__ __forceinline__ void set_range(Segment &g, int from, int64_t left) {
    const int to = (int)min((int64_t)places_of(g.steps), from + left);
    g.places = to - from;
    g.s0 = max(from - kPad, 0);
    g.s1 = max(to - kPad, 0);
}

// The segment that follows g on the line, with `left` places of the piece behind g.
__device__ __forceinline__ void next_segment(const PagedCache &c, int U, int parts, int64_t left, Segment &g) {
    if (++g.u == U) {
        g.u = 0;
        do {  // left > 0: a sequence with steps follows
            ++g.n;
            g.len = tokens_of(c, g.n);
        } while (g.len == 0);
        g.steps = (g.len + kStep - 1) / kStep;
    }
    g.head = parts == 1 ? g.u : g.u / parts;
    set_range(g, 0, left);
}

// Four channels of an output row (and the row's lse) from its sums.
template <int D>
__device__ __forceinline__ void write_row(const DecodeParams &p, int64_t row, int d, float4 a, float m, float sum) {
    const float inv = sum == 0.f ? 0.f : exp2_int(kRef - kTop) / sum;
    if (p.o_bf16) {
        uint2 w;
        w.x = pack_bf16x2(a.x * inv, a.y * inv);
        w.y = pack_bf16x2(a.z * inv, a.w * inv);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + row * D + d) = w;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + row * D + d) =
            make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    }
    if (p.lse && d == 0) p.lse[row] = sum == 0.f ? kNegInf : (log2f(sum) + m) * 0.6931471805599453f;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::CTAS) attn_decode_kernel(
    const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const __grid_constant__ DecodeParams p) {
    using F = Cfg<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ int64_t s_scan[kWarps];
    __shared__ Segment s_seg;
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.Hq / c.Hk, parts = (group + F::ROWS - 1) / F::ROWS, U = c.Hk * parts;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // this CTA's piece of the line
    int64_t L0 = 0, L1;
    if (p.whole) {
        Segment x;
        x.n = blockIdx.x / U;
        x.u = blockIdx.x - x.n * U;
        x.head = x.u / parts;
        x.len = tokens_of(c, x.n);
        x.steps = (x.len + kStep - 1) / kStep;
        L1 = places_of(x.steps);
        set_range(x, 0, L1);
        if (x.len == 0) {
            const int r0 = (x.u - x.head * parts) * F::ROWS;
            const int64_t row = (int64_t)x.n * p.Hq + x.head * group + r0;
            for (int i = tid; i < min(F::ROWS, group - r0) * D; i += kThreads) st_out(p.o, row * D + i, 0.f, p.o_bf16);
            if (p.lse && tid < min(F::ROWS, group - r0)) p.lse[row + tid] = kNegInf;
            return;
        }
        if (tid == 0) s_seg = x;
    } else {
        const Line line = measure_line(c, s_scan, kThreads);
        const int64_t all = line.total * U, S = piece_places(all, gridDim.x);
        L0 = (int64_t)blockIdx.x * S;
        if (L0 >= all) return;
        L1 = min(L0 + S, all);
        int64_t at = line.mine;  // one thread's range holds the start
        for (int n = line.first; n < line.last; ++n) {
            const int len = tokens_of(c, n), st = (len + kStep - 1) / kStep, pl = places_of(st);
            if (st > 0 && L0 >= at * U && L0 < (at + pl) * U) {
                const int64_t in = L0 - at * U;
                Segment x;
                x.n = n;
                x.len = len;
                x.steps = st;
                x.u = (int)(in / pl);
                x.head = x.u / parts;
                set_range(x, (int)(in - (int64_t)x.u * pl), L1 - L0);
                s_seg = x;
            }
            at += pl;
        }
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + F::BARS) + warp * F::DEPTH;  // this warp's slots
    if (lane == 0) {
        for (int i = 0; i < F::DEPTH; ++i) tc::mbar_init(bars + i, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    Segment cur = s_seg;

    // ---- the copying side: this warp's steps, F::DEPTH ahead
    const uint32_t ring = tc::smem_u32(smem) + warp * F::DEPTH * F::SLOT;
    const uint32_t scales_at = tc::smem_u32(smem) + F::SCALES + warp * F::DEPTH * 16;
    Segment ld = cur;
    int64_t ld_left = L1 - L0 - cur.places;  // of the piece, behind ld's segment
    int ld_s = ld.s0 + warp;
    bool ld_more = true;
    auto settle = [&] {  // moves on to the segment that holds this warp's next step
        while (ld_s >= ld.s1) {
            if (ld_left <= 0) {
                ld_more = false;
                return;
            }
            next_segment(c, U, parts, ld_left, ld);
            ld_left -= ld.places;
            ld_s = ld.s0 + warp;
        }
    };
    // A step's rows lie in one page, or with pages of 16 in two.  Lanes 0, 1 hold the first half's
    // page and fetch its two scales, lanes 2, 3 the second half's (-1 where there is none).
    const bool small = c.p_shift == 4;
    const int page_log = c.p_shift - 5, in_page = (1 << max(page_log, 0)) - 1;
    auto page_at = [&]() {
        const int half = lane >> 1;
        const int blk = small ? 2 * ld_s + half : ld_s >> page_log;
        return lane < 4 && (ld_s * 2 + half) * 16 < ld.len ? __ldg(c.block_table + (int64_t)ld.n * c.max_blocks + blk) : -1;
    };
    settle();
    int page = ld_more ? page_at() : -1;
    int wr = 0, issued = 0;
    int failed = 0;  // a copy's wait gave up: no further copies, NaN in what is left
    auto copy_step = [&] {
        if (ld_more && !failed) {
            const bool good = (uint32_t)page < (uint32_t)c.n_pages;
            const uint32_t slot = ring + wr * F::SLOT;
            if (lane < 4) {
                const uint32_t dst = scales_at + wr * 16 + lane * 4;
                if (good)
                    cp4(dst, ((lane & 1) ? c.v_scale : c.k_scale) + (int64_t)page * c.Hk + ld.head);
                else  // no such page: its tokens' scores are NaN, and so is the output
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(__int_as_float(0x7fc00000)) : "memory");
            }
            const int row = good ? ((int)(((int64_t)page * c.Hk + ld.head) << c.p_shift)) + (small ? 0 : (ld_s & in_page) << 5) : -1;
            const int row2 = __shfl_sync(0xffffffffu, row, 2);
            if (lane == 0) {
                const int rows = (row >= 0 ? small ? 16 : 32 : 0) + (small && row2 >= 0 ? 16 : 0);
                tc::mbar_arrive_expect_tx(bars + wr, rows * 2 * D);
                if (row >= 0) {
                    tc::tma_load_2d(slot, &map_k, bars + wr, 0, row);
                    tc::tma_load_2d(slot + F::KBYTES, &map_v, bars + wr, 0, row);
                }
                if (small && row2 >= 0) {
                    tc::tma_load_2d(slot + F::HALF, &map_k, bars + wr, 0, row2);
                    tc::tma_load_2d(slot + F::KBYTES + F::HALF, &map_v, bars + wr, 0, row2);
                }
            }
            ++issued;
            ld_s += kWarps;
            if (ld_s >= ld.s1) settle();
            if (ld_more) page = page_at();  // the next step's page number is on its way meanwhile
            wr = wr + 1 == F::DEPTH ? 0 : wr + 1;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < F::DEPTH; ++i) copy_step();

    // ---- the computing side
    float *merge = reinterpret_cast<float *>(smem + F::MERGE);  // [2][row][PITCH] sums, then M and l
    float *merge_m = merge + 2 * F::ROWS * F::PITCH, *merge_l = merge_m + 2 * F::ROWS;
    const float log2e_scale = p.scale * 1.4426950408889634f;
    int64_t left = L1 - L0;
    // where this lane's pieces of a step lie: 16-byte piece x of row r is at x ^ (r % 8) of its 128
    // bytes, or at x ^ (r / 2 % 4) of 64
    const int k_at[2] = {D == 128 ? g * 128 + (((2 * t) ^ g) << 4) : g * 64 + ((t ^ (g >> 1)) << 4),
                         g * 128 + (((2 * t + 1) ^ g) << 4)};
    const int v_at[2] = {D == 128 ? 2 * t * 128 + ((g ^ (2 * t)) << 4) : 2 * t * 64 + (((g >> 1) ^ t) << 4) + 8 * (g & 1),
                         D == 128 ? (2 * t + 1) * 128 + ((g ^ (2 * t + 1)) << 4)
                                  : (2 * t + 1) * 64 + (((g >> 1) ^ t) << 4) + 8 * (g & 1)};
    int rd = 0, odd = 0;
    uint32_t rd_phase = 0;
    bool first = true;
    // A unit's queries: each lane the 16-byte pieces of its row that its products take.
    uint4 qw[NT][F::KJ][2];
    auto fetch_queries = [&](const Segment &x) {
        const int r0 = (x.u - x.head * parts) * F::ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = r0 + nt * 8 + g;
            const __nv_bfloat16 *q = p.q + x.n * p.q_stride + (int64_t)(x.head * group + r) * D;
#pragma unroll
            for (int j = 0; j < F::KJ; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qw[nt][j][i] = r < group ? __ldg(reinterpret_cast<const uint4 *>(q + 16 * (F::KJ * t + j) + 8 * i))
                                             : make_uint4(0, 0, 0, 0);
        }
    };
    fetch_queries(cur);
    while (true) {
        const int h = cur.head, r0 = (cur.u - h * parts) * F::ROWS;  // first query head of the unit in its group
        // queries: f16, each row scaled by a power of two so that its largest lies in [2^14, 2^15): nothing
        // overflows, and what lies up to 2^31 below it is exact (8 bits down to 2^-24, the least f16 number)
        uint32_t qf[NT][F::KJ * 4][2];
        float row_scale[NT][2];  // of the two rows whose scores this lane holds
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < F::KJ; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 w = qw[nt][j][i];
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = (u[e] << 16) & 0x7FFF0000u, hi = u[e] & 0x7FFF0000u;
                        if (lo < 0x7F800000u) amax = max(amax, lo);
                        if (hi < 0x7F800000u) amax = max(amax, hi);
                    }
                }
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int e = max((int)(amax >> 23) - 127, -100) - 14;
            const float inv = exp2_int(-e);
#pragma unroll
            for (int j = 0; j < F::KJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = qw[nt][j][i >> 1];
                    const uint32_t lo = (i & 1) ? x.z : x.x, hi = (i & 1) ? x.w : x.y;
                    qf[nt][4 * j + i][0] = pack_half(__uint_as_float(lo << 16) * inv, __uint_as_float(lo & 0xFFFF0000u) * inv);
                    qf[nt][4 * j + i][1] = pack_half(__uint_as_float(hi << 16) * inv, __uint_as_float(hi & 0xFFFF0000u) * inv);
                }
            const float rs = log2e_scale * exp2_int(e);
            row_scale[nt][0] = __shfl_sync(0xffffffffu, rs, (2 * t) * 4);
            row_scale[nt][1] = __shfl_sync(0xffffffffu, rs, (2 * t + 1) * 4);
        }

        float acc[NT][F::MT][4] = {};
        float M[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            M[nt][0] = M[nt][1] = kNegInf;
            l[nt][0] = l[nt][1] = 0.f;
        }
        for (int s = cur.s0 + warp; s < cur.s1; s += kWarps) {
            cp_wait<F::DEPTH - 1>();
            if (!failed && !tc::mbar_wait(bars + rd, rd_phase, p.polls)) failed = 1;
            failed = __any_sync(0xffffffffu, failed);
            __syncwarp();  // the scales came by four lanes' own copies; a vote orders no memory
            const uint8_t *slot = smem + (warp * F::DEPTH + rd) * F::SLOT;
            const float4 sc = *reinterpret_cast<const float4 *>(smem + F::SCALES + (warp * F::DEPTH + rd) * 16);
            const float ks[2] = {sc.x, sc.z}, vs[2] = {sc.y, sc.w};
            float S[2][NT][4] = {};
#pragma unroll
            for (int j = 0; j < F::KJ; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(slot + h * F::HALF + k_at[j]);
                    const uint4 b = *reinterpret_cast<const uint4 *>(slot + h * F::HALF + F::HALF / 2 + k_at[j]);
                    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t a0, a1, a2, a3;
                        widen(wa[i], a0, a2);
                        widen(wb[i], a1, a3);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_f16(S[h][nt], a0, a1, a2, a3, qf[nt][4 * j + i][0], qf[nt][4 * j + i][1]);
                    }
                }
            const bool tail = (s + 1) * kStep > cur.len;  // places behind the last token
            bool over = false;
            float ev[2];  // reference of the value scale: its binary exponent
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int be = (int)(__float_as_uint(vs[h]) >> 23) & 0xFF;
                ev[h] = (float)(be == 0xFF ? 0 : max(be - 127, kLeastScale));  // a NaN moves nothing
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float c0 = row_scale[nt][0] * ks[h], c1 = row_scale[nt][1] * ks[h];
                    S[h][nt][0] *= c0;
                    S[h][nt][1] *= c1;
                    S[h][nt][2] *= c0;
                    S[h][nt][3] *= c1;
                }
                if (tail) {
                    const int tok = s * kStep + 16 * h + g;
                    if (s * kStep + 16 * h >= cur.len) ev[h] = kNegInf;  // this half's scales stand for nothing
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        S[h][nt][0] = tok < cur.len ? S[h][nt][0] : kNegInf;
                        S[h][nt][1] = tok < cur.len ? S[h][nt][1] : kNegInf;
                        S[h][nt][2] = tok + 8 < cur.len ? S[h][nt][2] : kNegInf;
                        S[h][nt][3] = tok + 8 < cur.len ? S[h][nt][3] : kNegInf;
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    over |= fmaxf(S[h][nt][0], S[h][nt][2]) > M[nt][0] + (kRef + kSlack - ev[h]) ||
                            fmaxf(S[h][nt][1], S[h][nt][3]) > M[nt][1] + (kRef + kSlack - ev[h]);
            }
            if (__any_sync(0xffffffffu, over)) {  // raise the maximum and bring the sums to it
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(fmaxf(S[0][nt][e], S[0][nt][e + 2]) + ev[0], fmaxf(S[1][nt][e], S[1][nt][e + 2]) + ev[1]);
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m - kRef, M[nt][e]);
                        const float f = root_factor(M[nt][e], m);
                        M[nt][e] = m;
                        l[nt][e] = bring(l[nt][e], f);
#pragma unroll
                        for (int j = 0; j < F::MT; ++j) {
                            acc[nt][j][e] = bring(acc[nt][j][e], f);
                            acc[nt][j][e + 2] = bring(acc[nt][j][e + 2], f);
                        }
                    }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t x[NT][2];
                const float vscale = tail && s * kStep + 16 * h >= cur.len ? 0.f : vs[h] * exp2_int(kTop - kRef);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float m0 = M[nt][0] == kNegInf ? 0.f : M[nt][0], m1 = M[nt][1] == kNegInf ? 0.f : M[nt][1];
                    const float e0 = ex2(S[h][nt][0] - m0), e1 = ex2(S[h][nt][1] - m1), e2 = ex2(S[h][nt][2] - m0),
                                e3 = ex2(S[h][nt][3] - m1);
                    l[nt][0] += e0 + e2;
                    l[nt][1] += e1 + e3;
                    x[nt][0] = pack_half(e0 * vscale, e1 * vscale);
                    x[nt][1] = pack_half(e2 * vscale, e3 * vscale);
                }
                add_products<D, NT, false>(acc, x, slot + F::KBYTES + h * F::HALF, v_at[0], v_at[1],
                                           tail ? cur.len - s * kStep - 16 * h : 16);
            }
            if (++rd == F::DEPTH) rd = 0, rd_phase ^= 1;
            __syncwarp();  // every lane has read the slot: it is filled again
            copy_step();
        }
        {
            // f16 takes 2^-25 at most from a weight below 2^-14, and a value's code is at most 448: over this warp's
            // tokens, as many as 128 times `enough` says, less than 2^-9 (half a step of bf16) of `enough`.  (Most
            // codes are far smaller; with a quarter of this, values of 0.05 under a scale of one sent long
            // sequences through their steps twice, 268 us for 113.)
            const float enough = 0.25f * (float)((cur.s1 - cur.s0) / kWarps + 1);
            float sums = INFINITY;  // the least row's largest sum among this lane's channels
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float a = 0.f;
#pragma unroll
                    for (int j = 0; j < F::MT; ++j) a = fmaxf(fmaxf(a, fabsf(acc[nt][j][e])), fabsf(acc[nt][j][e + 2]));
                    sums = fminf(sums, a);
                }
            if (__any_sync(0xffffffffu, sums < enough) && cur.s0 + warp < cur.s1 && !failed) {
                Again<D, NT> x;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < F::KJ * 4; ++i) x.q[nt][i][0] = qf[nt][i][0], x.q[nt][i][1] = qf[nt][i][1];
#pragma unroll
                    for (int e = 0; e < 2; ++e) x.row_scale[nt][e] = row_scale[nt][e], x.M[nt][e] = M[nt][e];
                }
                again_with_rest<D, NT>(p, cur.n, cur.head, cur.len, cur.s0 + warp, cur.s1, x);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < F::MT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[nt][j][e] = x.acc[nt][j][e];
            }
        }
        if (failed) {  // a copy's wait gave up: the sums stand for nothing
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) l[nt][0] = l[nt][1] = __int_as_float(0x7fc00000);
        }

        // the next unit and its queries, on their way while this one's sums come together
        left -= cur.places;
        Segment nxt = cur;
        if (left > 0) {
            next_segment(c, U, parts, left, nxt);
            fetch_queries(nxt);
        }

        // ---- the warps' sums of this unit together: one pair of warps leaves its sums and goes on with the
        // next unit, the other adds them to its own, and then the two of those.  The pairs change
        // parts from unit to unit, so the buffer's last readers are the next to fill it.
        if (cur.s1 > cur.s0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
                    x += __shfl_xor_sync(0xffffffffu, x, 4);
                    x += __shfl_xor_sync(0xffffffffu, x, 8);
                    x += __shfl_xor_sync(0xffffffffu, x, 16);
                    l[nt][e] = x;
                }
            float *buf = merge + (warp & 1) * F::ROWS * F::PITCH + g * F::VB;
            float *buf_m = merge_m + (warp & 1) * F::ROWS, *buf_l = merge_l + (warp & 1) * F::ROWS;
            auto put = [&] {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = nt * 8 + 2 * t + e;
                        if (g == 0) {
                            buf_m[r] = M[nt][e];
                            buf_l[r] = l[nt][e];
                        }
#pragma unroll
                        for (int j = 0; j < F::MT; ++j)
                            *reinterpret_cast<float2 *>(buf + r * F::PITCH + 2 * j) = make_float2(acc[nt][j][e], acc[nt][j][e + 2]);
                    }
            };
            const bool leaves = (warp >> 1) == (odd ? 0 : 1);
            const int pair = 3 + (warp >> 1), filled = 1 + odd;
            odd ^= 1;
            bar_sync(pair, 64);  // both have read what they left here last
            if (leaves) {
                put();
                bar_arrive(filled, kThreads);
            } else {
                bar_sync(filled, kThreads);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = nt * 8 + 2 * t + e;
                        const float mo = buf_m[r], m = fmaxf(M[nt][e], mo);
                        const float fa = root_factor(M[nt][e], m), fb = root_factor(mo, m);
                        M[nt][e] = m;
                        l[nt][e] = bring(l[nt][e], fa) + bring(buf_l[r], fb);
#pragma unroll
                        for (int j = 0; j < F::MT; ++j) {
                            const float2 x = *reinterpret_cast<const float2 *>(buf + r * F::PITCH + 2 * j);
                            acc[nt][j][e] = bring(acc[nt][j][e], fa) + bring(x.x, fb);
                            acc[nt][j][e + 2] = bring(acc[nt][j][e + 2], fa) + bring(x.y, fb);
                        }
                    }
                __syncwarp();  // every lane has read M and l
                put();
                bar_sync(pair, 64);
                const bool whole = cur.s0 == 0 && cur.s1 == cur.steps;
                float *part = p.ws + ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * F::PART;
                for (int i = tid & 63; i < F::ROWS * (D / 4); i += 64) {
                    const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
                    const float ma = merge_m[r], mb = merge_m[F::ROWS + r], m = fmaxf(ma, mb);
                    const float fa = root_factor(ma, m), fb = root_factor(mb, m);
                    const float4 x = *reinterpret_cast<const float4 *>(merge + r * F::PITCH + d);
                    const float4 y = *reinterpret_cast<const float4 *>(merge + (F::ROWS + r) * F::PITCH + d);
                    const float4 a = make_float4(bring(x.x, fa) + bring(y.x, fb), bring(x.y, fa) + bring(y.y, fb),
                                                 bring(x.z, fa) + bring(y.z, fb), bring(x.w, fa) + bring(y.w, fb));
                    const float sum = bring(merge_l[r], fa) + bring(merge_l[F::ROWS + r], fb);
                    if (!whole) {
                        *reinterpret_cast<float4 *>(part + r * D + d) = a;
                        if (d == 0) {
                            part[F::ROWS * D + r] = m;
                            part[F::ROWS * D + F::ROWS + r] = sum;
                        }
                    } else if (r0 + r < group) {
                        write_row<D>(p, (int64_t)cur.n * p.Hq + h * group + r0 + r, d, a, m, sum);
                    }
                }
            }
        }
        first = false;
        if (left <= 0) break;
        cur = nxt;
    }
    cp_wait<0>();
    // after a failure copies may still be under way: they land before the CTA ends
    if (failed) {
        for (int i = max(0, issued - F::DEPTH); i < issued; ++i) tc::mbar_wait(bars + i % F::DEPTH, (i / F::DEPTH) & 1, kAttnPolls);
        if (lane == 0) atomicAdd(&g_attn_decode_timeouts, 1);
    }
}

// Joins the units that more than one CTA took, adding their pieces in their order along the
// line; gridDim.y CTAs share a unit's rows, and the runs of a CTA's threads its pieces.  With
// at least as many CTAs as units blockIdx.x is the unit; else it is a piece, and the CTA
// looks after the unit that begins in it and goes on behind it, if there is one.  (A CTA for
// every query row of the batch, most of which had nothing to do, took 17 us of 118 with 256
// sequences.)  Rows of sequences without tokens are written here as zero.
template <int D, int NT>
__global__ void __launch_bounds__(kJoinMost) attn_decode_join_kernel(const __grid_constant__ DecodeParams p, int ctas,
                                                                     int by_unit) {
    using F = Cfg<D, NT>;
    __shared__ int64_t s_scan[kJoinMost / 32];
    __shared__ int64_t s_begin;
    __shared__ Segment s_seg;
    __shared__ float4 s_acc[kJoinMost];
    __shared__ float s_m[kJoinMost], s_l[kJoinMost];
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, group = p.Hq / c.Hk, parts = (group + F::ROWS - 1) / F::ROWS, U = c.Hk * parts;
    const int rows = F::ROWS / gridDim.y, items = rows * (D / 4), groups = blockDim.x / items;  // four channels an item
    const Line line = measure_line(c, s_scan, blockDim.x);
    const int64_t all = line.total * U, S = piece_places(all, ctas), L0 = (int64_t)blockIdx.x * S, L1 = min(L0 + S, all);
    if (tid == 0) s_seg.n = -1;
    __syncthreads();
    if (by_unit || L0 < L1) {
        const int un = blockIdx.x / U;  // by_unit: the unit's sequence
        int64_t at = line.mine;
        for (int n = line.first; n < line.last; ++n) {
            const int st = steps_of(c, n), pl = places_of(st);
            if (st > 0 && (by_unit ? n == un : L1 - 1 >= at * U && L1 - 1 < (at + pl) * U)) {
                s_seg.u = by_unit ? blockIdx.x - un * U : (int)((L1 - 1 - at * U) / pl);
                s_seg.steps = st;
                s_seg.n = n;
                s_begin = at * U + (int64_t)s_seg.u * pl;
            }
            at += pl;
        }
    }
    __syncthreads();
    const int n = s_seg.n, u = s_seg.u, steps = s_seg.steps;
    const int64_t begin = s_begin;  // of the unit, on the line
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.y == gridDim.y - 1)
        for (int e = blockIdx.x; e < c.N; e += gridDim.x) {
            if (tokens_of(c, e) > 0) continue;
            const int64_t row = (int64_t)e * p.Hq;
            for (int i = tid; i < p.Hq * D; i += blockDim.x) st_out(p.o, row * D + i, 0.f, p.o_bf16);
            if (p.lse)
                for (int i = tid; i < p.Hq; i += blockDim.x) p.lse[row + i] = kNegInf;
        }
    if (n < 0) return;
    const int64_t c0 = (begin + kPad) / S, c1 = (begin + kPad + steps - 1) / S;  // CTAs of its first and last step
    if (c1 == c0 || (!by_unit && c0 != blockIdx.x)) return;
    const int item = tid % items, r = rows * blockIdx.y + item / (D / 4), d = item % (D / 4) * 4;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = kNegInf, l = 0.f;
    const int pieces = (int)(c1 - c0) + 1, used = min(groups, pieces), per = (pieces + used - 1) / used;
    const int64_t k0 = c0 + (int64_t)(tid / items) * per, k1 = min(k0 + per, c1 + 1);
#pragma unroll 4
    for (int64_t k = k0; k < k1; ++k) {
        // the unit is the first of its CTA's segments unless the CTA began before it
        const float *part = p.ws + (k * 2 + (k * S >= begin ? 0 : 1)) * F::PART;
        const float mk = __ldcg(part + F::ROWS * D + r), lk = __ldcg(part + F::ROWS * D + F::ROWS + r);
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(part + r * D + d));
        const float mn = fmaxf(m, mk);
        const float f = root_factor(m, mn), fk = root_factor(mk, mn);
        m = mn;
        l = bring(l, f) + bring(lk, fk);
        a = make_float4(bring(a.x, f) + bring(x.x, fk), bring(a.y, f) + bring(x.y, fk), bring(a.z, f) + bring(x.z, fk),
                        bring(a.w, f) + bring(x.w, fk));
    }
    s_acc[tid] = a;
    s_m[tid] = m;
    s_l[tid] = l;
    __syncthreads();
    const int h = parts == 1 ? u : u / parts, head = (u - h * parts) * F::ROWS + r;  // within the group
    if (tid >= items || head >= group) return;
    for (int i = 1; i < used; ++i) m = fmaxf(m, s_m[tid + i * items]);
    float sum = 0.f;
    a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < used; ++i) {
        const float f = root_factor(s_m[tid + i * items], m);
        const float4 x = s_acc[tid + i * items];
        sum += bring(s_l[tid + i * items], f);
        a = make_float4(a.x + bring(x.x, f), a.y + bring(x.y, f), a.z + bring(x.z, f), a.w + bring(x.w, f));
    }
    write_row<D>(p, (int64_t)n * p.Hq + h * group + head, d, a, m, sum);
}

// The cache's rows (D bytes each) in boxes of a step's rows, or of a page's where those are fewer.
bool encode(chunk::EncodeTiledFn enc, CUtensorMap *map, const void *base, const PagedCache &c) {
    const cuuint64_t dims[2] = {(cuuint64_t)c.D, (cuuint64_t)c.n_pages * c.Hk * c.P};
    const cuuint64_t strides[1] = {(cuuint64_t)c.D};
    const cuuint32_t box[2] = {(cuuint32_t)c.D, (cuuint32_t)(c.P < kStep ? c.P : kStep)}, es[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) set_error("attn_decode: cuTensorMapEncodeTiled failed (%d)", (int)r);
    return r == CUDA_SUCCESS;
}

// CTAs of a call: what the GPU holds at once, or as many as pieces are possible at all.  Where the
// table holds few tokens, heads are not cut, each has a CTA, and nothing is joined: cut and
// whole, 32/8 heads of 128, one sequence of 60, 500 tokens 6.5 and 4.5, 9.0 and 8.2 us (1000: 8.8
// and 12.3 when the rule was made); 32 of 250, 1000 tokens 12.3 and 7.5, 22.2 and 17.8 us; 256 of
// [50, 150], [900, 1000] with 64/8 heads 35.0 and 30.4, 93.9 and 93.4 us.  With groups of 16, where
// an SM holds two CTAs, many waves of them are slower: 64 sequences of 500 tokens 32.7 and 29.8,
// 256 82.5 and 87.7 us when the rule was made.
template <int D, int NT>
int decode_ctas(int64_t N, int Hq, int Hk, int64_t max_tokens, bool &whole) {
    using F = Cfg<D, NT>;
    const int64_t most = (int64_t)F::CTAS * sm_count(), group = Hq / Hk;
    const int64_t units = N * Hk * ((group + F::ROWS - 1) / F::ROWS);
    whole = max_tokens <= (2 * units >= most ? 32 : 16) * kStep && units <= (NT == 1 ? INT32_MAX : 2 * most);
    if (whole) return (int)units;
    const int64_t pieces = (units * ((max_tokens + kStep - 1) / kStep + kPad) + kMinPiece - 1) / kMinPiece;
    return (int)(pieces < most ? pieces : most);
}

template <int D, int NT>
size_t workspace_bytes(int64_t N, int Hq, int Hk, int64_t max_tokens) {
    bool whole;
    const int ctas = decode_ctas<D, NT>(N, Hq, Hk, max_tokens, whole);
    return whole ? 0 : (size_t)ctas * 2 * Cfg<D, NT>::PART * sizeof(float);  // two pieces per CTA
}

template <int D, int NT>
kda_status run(const DecodeParams &p, cudaStream_t st) {
    using F = Cfg<D, NT>;
    chunk::EncodeTiledFn enc = reinterpret_cast<chunk::EncodeTiledFn>(tensor_map_encoder());
    if (!enc) {
        set_error("attn_decode: cuTensorMapEncodeTiled is not available from the driver");
        return KDA_ERR_CUDA;
    }
    CUtensorMap mk, mv;
    if (!encode(enc, &mk, p.c.k, p.c) || !encode(enc, &mv, p.c.v, p.c)) return KDA_ERR_CUDA;
    static DeviceOnce configured;
    bool whole;
    const int dev = current_device();
    const int ctas = decode_ctas<D, NT>(p.c.N, p.Hq, p.c.Hk, (int64_t)p.c.max_blocks * p.c.P, whole);
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(attn_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM) !=
            cudaSuccess) {
            set_error("attn_decode: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    DecodeParams call = p;
    call.whole = whole;
    attn_decode_kernel<D, NT><<<ctas, kThreads, F::SMEM, st>>>(mk, mv, call);
    note_launch();
    kda_status s = check_launch("attn_decode_kernel");
    if (whole || s != KDA_OK) return s;
    cudaLaunchConfig_t cfg = {};
    // few units (of which each may have many pieces): large CTAs for two rows each; else as many
    // as are resident at once, so that none waits for others that wait for the first kernel
    const int group = p.Hq / p.c.Hk, units = p.c.N * p.c.Hk * ((group + F::ROWS - 1) / F::ROWS);
    const bool few = (int64_t)units * (F::ROWS / 2) <= 4 * sm_count();
    cfg.gridDim = dim3(units < ctas ? units : ctas, few ? F::ROWS / 2 : 2, 1);
    cfg.blockDim = dim3(few ? 512 : 256, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // starts while the first kernel ends; waits for it before it reads
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, NT>, p, ctas, units < ctas ? 1 : 0);
    note_launch();
    if (e != cudaSuccess) {
        set_error("attn_decode_join_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return check_launch("attn_decode_join_kernel");
}

}  // namespace

int take_attn_decode_timeouts(cudaStream_t st) {
    int n = 0;
    const int zero = 0;
    if (cudaMemcpyFromSymbolAsync(&n, g_attn_decode_timeouts, sizeof(int), 0, cudaMemcpyDeviceToHost, st) !=
            cudaSuccess ||
        cudaMemcpyToSymbolAsync(g_attn_decode_timeouts, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st) !=
            cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess) {
        set_error("attn_decode: cannot read the timeout counter: %s", cudaGetErrorString(cudaGetLastError()));
        return -1;
    }
    return n;
}

size_t attn_decode_workspace_bytes(int64_t N, int Hq, int Hk, int D, int64_t max_tokens) {
    const bool wide = Hq / Hk > 8;
    if (D == 128) return wide ? workspace_bytes<128, 2>(N, Hq, Hk, max_tokens) : workspace_bytes<128, 1>(N, Hq, Hk, max_tokens);
    return wide ? workspace_bytes<64, 2>(N, Hq, Hk, max_tokens) : workspace_bytes<64, 1>(N, Hq, Hk, max_tokens);
}

kda_status launch_attn_decode(const DecodeParams &p, cudaStream_t st) {
    if (p.c.N == 0) return KDA_OK;
    const bool wide = p.Hq / p.c.Hk > 8;
    if (p.c.D == 128) return wide ? run<128, 2>(p, st) : run<128, 1>(p, st);
    return wide ? run<64, 2>(p, st) : run<64, 1>(p, st);
}

}  // namespace kda
