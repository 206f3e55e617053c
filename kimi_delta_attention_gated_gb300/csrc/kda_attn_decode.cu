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
// The value scale is folded into P: with M >= max_j (s_j + log2 vs_j), e_j = 2^(s_j - M) is
// summed for the denominator and e_j * vs_j <= 2^kSlack is rounded to f16 for the product,
// so pages of very different scales share one accumulator.
//
// Work split.  All (sequence, head, 16 tokens) steps are numbered in one line, and the line
// is cut into equal pieces, one per CTA, whatever the lengths of the sequences are; every
// CTA finds its piece from the lengths on the device.  A head that one CTA covers is written
// at once, the others go through a workspace and attn_decode_join_kernel, which adds a
// head's pieces in their order, so results do not depend on timing.
//
// Copies.  Each lane copies exactly the bytes it will use (cp.async) into a ring of its own
// in shared memory, kDepth steps ahead and across the borders of heads: no barrier and no
// bank conflict between the copy and its use.
#include <cuda_fp16.h>

#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;       // tokens of a step
constexpr int kDepth = 3;       // steps in flight per warp
constexpr int kMinSteps = 8;    // steps of a CTA at least
constexpr float kSlack = 8.f;   // the maximum in use may lie this far below the true one (log2)
constexpr int kCtasPerSm = 3;
constexpr float kNegInf = -INFINITY;

template <int D, int NT>
struct Cfg {
    static constexpr int ROWS = 8 * NT;                 // query heads of a unit
    static constexpr int KJ = D / 64;                   // 64-byte pieces of a key row
    static constexpr int VB = D / 8;                    // bytes of a value row per lane
    static constexpr int MT = D / 16;                   // 16-channel tiles of the output
    static constexpr int KBYTES = kStep * D, VBYTES = kStep * D;
    static constexpr int SLOT = KBYTES + VBYTES + 16;   // + the two scales
    static constexpr int PITCH = D + 4;                 // fp32 row of the merge buffer
    static constexpr int RING = kWarps * kDepth * SLOT;
    static constexpr int MERGE = kWarps * ROWS * (PITCH + 2) * 4;
    static constexpr int SMEM = RING + MERGE;
    static constexpr int PART = ROWS * (D + 2);         // floats of one piece in the workspace
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two e4m3 codes (the low / high half of w) as f16.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    return (uint32_t)h.x | (uint32_t)h.y << 16;
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

// Tokens and steps of sequence n, its length clamped to what its block table can hold.
__device__ __forceinline__ int tokens_of(const PagedCache &c, int n) {
    const int64_t room = (int64_t)c.max_blocks * c.P;
    return (int)max((int64_t)0, min((int64_t)c.lens[n], min(room, (int64_t)INT32_MAX - kStep)));
}
__device__ __forceinline__ int steps_of(const PagedCache &c, int n) { return (tokens_of(c, n) + kStep - 1) / kStep; }

// The line of steps: sequence n's U units (head, part of its group) lie one after another,
// each steps_of(n) long, behind those of the sequences before.  Returns the steps of all
// sequences (of one unit each) to every thread, and this thread's share of the prefix.
struct Line {
    int64_t total;  // steps of all sequences, one unit each
    int64_t mine;   // those before this thread's first sequence
    int first, last;  // this thread's sequences [first, last)
};
__device__ __forceinline__ Line measure_line(const PagedCache &c, int64_t *scan) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (c.N + kThreads - 1) / kThreads;
    Line l;
    l.first = min(tid * per, c.N);
    l.last = min(l.first + per, c.N);
    int64_t own = 0;
    for (int n = l.first; n < l.last; ++n) own += steps_of(c, n);
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
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) l.mine += scan[w];
        l.total += scan[w];
    }
    return l;
}
__device__ __forceinline__ int64_t piece_steps(int64_t line, int ctas) {
    const int64_t s = (line + ctas - 1) / ctas;
    return s < kMinSteps ? kMinSteps : s;
}

// A run of steps within one unit: [s0, s1) of unit u of sequence n.
struct Segment {
    int n, u, steps, len;
    int s0, s1;
};

// The segment that follows g on the line, with `left` steps of the piece behind it.
__device__ __forceinline__ void next_segment(const PagedCache &c, int U, int64_t left, Segment &g) {
    if (++g.u == U) {
        g.u = 0;
        do {  // left > 0: a sequence with steps follows
            ++g.n;
            g.len = tokens_of(c, g.n);
        } while (g.len == 0);
        g.steps = (g.len + kStep - 1) / kStep;
    }
    g.s0 = 0;
    g.s1 = (int)min((int64_t)g.steps, left);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) attn_decode_kernel(const __grid_constant__ DecodeParams p) {
    using F = Cfg<D, NT>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t s_scan[kWarps];
    __shared__ Segment s_seg;
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = p.Hq / c.Hk, parts = (group + F::ROWS - 1) / F::ROWS, U = c.Hk * parts;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // this CTA's piece of the line
    const Line line = measure_line(c, s_scan);
    const int64_t steps_all = line.total * U, S = piece_steps(steps_all, gridDim.x), L0 = (int64_t)blockIdx.x * S;
    if (L0 >= steps_all) return;
    const int64_t L1 = min(L0 + S, steps_all);
    {
        int64_t at = line.mine;  // one thread's range holds the start
        for (int n = line.first; n < line.last; ++n) {
            const int len = tokens_of(c, n), st = (len + kStep - 1) / kStep;
            if (st > 0 && L0 >= at * U && L0 < (at + st) * U) {
                const int64_t in = L0 - at * U;
                Segment x;
                x.n = n;
                x.len = len;
                x.steps = st;
                x.u = (int)(in / st);
                x.s0 = (int)(in - (int64_t)x.u * st);
                x.s1 = (int)min((int64_t)st, x.s0 + (L1 - L0));
                s_seg = x;
            }
            at += st;
        }
    }
    __syncthreads();
    Segment cur = s_seg;

    // ---- the copying side: this warp's steps, kDepth ahead
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kDepth * F::SLOT;
    Segment ld = cur;
    int64_t ld_left = L1 - L0 - (cur.s1 - cur.s0);  // steps of the piece behind ld's segment
    int ld_s = ld.s0 + warp;
    bool ld_more = true;
    auto settle = [&] {  // moves on to the segment that holds this warp's next step
        while (ld_s >= ld.s1) {
            if (ld_left <= 0) {
                ld_more = false;
                return;
            }
            next_segment(c, U, ld_left, ld);
            ld_left -= ld.s1 - ld.s0;
            ld_s = ld.s0 + warp;
        }
    };
    auto page_at = [&]() { return __ldg(c.block_table + (int64_t)ld.n * c.max_blocks + ld_s * kStep / c.P); };
    settle();
    int page = ld_more ? page_at() : 0;
    int wr = 0;
    auto copy_step = [&] {
        if (ld_more) {
            const uint32_t slot = ring + wr * F::SLOT;
            const bool good = page >= 0 && page < c.n_pages;
            const int64_t blk = (int64_t)(good ? page : 0) * c.Hk + ld.u / parts;
            const int tok0 = ld_s * kStep, valid = good ? ld.len - tok0 : 0;  // tokens of the step that exist
            const int64_t base = (blk * c.P + tok0 % c.P) * D;
            const uint8_t *k = c.k + base, *v = c.v + base;
#pragma unroll
            for (int j = 0; j < F::KJ; ++j) {
                cp16(slot + (2 * j) * 512 + lane * 16, k + g * D + 64 * j + 16 * t, g < valid ? 16 : 0);
                cp16(slot + (2 * j + 1) * 512 + lane * 16, k + (g + 8) * D + 64 * j + 16 * t, g + 8 < valid ? 16 : 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = 2 * t + (i & 1) + (i >> 1) * 8;
                const uint32_t dst = slot + F::KBYTES + i * (32 * F::VB) + lane * F::VB;
                if (F::VB == 16)
                    cp16(dst, v + tok * D + 16 * g, tok < valid ? 16 : 0);
                else
                    cp8(dst, v + tok * D + 8 * g, tok < valid ? 8 : 0);
            }
            if (lane < 2) {
                const uint32_t dst = slot + F::KBYTES + F::VBYTES + lane * 4;
                if (good)
                    cp4(dst, (lane ? c.v_scale : c.k_scale) + blk);
                else  // no such page: its tokens' scores are NaN, and so is the output
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(dst), "f"(__int_as_float(0x7fc00000)) : "memory");
            }
            ld_s += kWarps;
            settle();
            if (ld_more) page = page_at();  // the next step's page number is on its way meanwhile
            wr = wr + 1 == kDepth ? 0 : wr + 1;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth - 1; ++i) copy_step();

    // ---- the computing side
    float *merge = reinterpret_cast<float *>(smem + F::RING);  // [warp][row][PITCH] sums, then M and l
    float *merge_m = merge + kWarps * F::ROWS * F::PITCH, *merge_l = merge_m + kWarps * F::ROWS;
    const float log2e_scale = p.scale * 1.4426950408889634f;
    int64_t left = L1 - L0;
    int rd = 0;
    bool first = true;
    while (true) {
        const int h = cur.u / parts, r0 = (cur.u - h * parts) * F::ROWS;  // first query head of the unit in its group
        // queries: f16, each row scaled by a power of two to at most 2 so that nothing overflows
        uint32_t qf[NT][F::KJ * 4][2];
        float row_scale[NT][2];  // of the two rows whose scores this lane holds
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = r0 + nt * 8 + g;
            const __nv_bfloat16 *q = p.q + cur.n * p.q_stride + (int64_t)(h * group + r) * D;
            uint4 w[F::KJ][2];
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < F::KJ; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[j][i] = r < group ? __ldg(reinterpret_cast<const uint4 *>(q + 64 * j + 16 * t + 8 * i))
                                        : make_uint4(0, 0, 0, 0);
                    const uint32_t u[4] = {w[j][i].x, w[j][i].y, w[j][i].z, w[j][i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t lo = (u[e] << 16) & 0x7FFF0000u, hi = u[e] & 0x7FFF0000u;
                        if (lo < 0x7F800000u) amax = max(amax, lo);
                        if (hi < 0x7F800000u) amax = max(amax, hi);
                    }
                }
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            const int e = min(max((int)(amax >> 23) - 127, -100), 126);
            const float inv = exp2_int(-e);
#pragma unroll
            for (int j = 0; j < F::KJ; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 x = w[j][i >> 1];
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
            copy_step();
            cp_wait<kDepth - 1>();
            __syncwarp();
            const uint8_t *slot = smem + (warp * kDepth + rd) * F::SLOT;
            rd = rd + 1 == kDepth ? 0 : rd + 1;
            const float2 sc = *reinterpret_cast<const float2 *>(slot + F::KBYTES + F::VBYTES);
            float S[NT][4] = {};
#pragma unroll
            for (int j = 0; j < F::KJ; ++j) {
                const uint4 a = *reinterpret_cast<const uint4 *>(slot + (2 * j) * 512 + lane * 16);
                const uint4 b = *reinterpret_cast<const uint4 *>(slot + (2 * j + 1) * 512 + lane * 16);
                const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a0 = widen_lo(wa[i]), a1 = widen_lo(wb[i]), a2 = widen_hi(wa[i]), a3 = widen_hi(wb[i]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(S[nt], a0, a1, a2, a3, qf[nt][4 * j + i][0], qf[nt][4 * j + i][1]);
                }
            }
            const int tok0 = s * kStep;
            const bool in0 = tok0 + g < cur.len, in1 = tok0 + g + 8 < cur.len;
            // reference of the value scale: its binary exponent
            const float ev = (float)((int)((__float_as_uint(sc.y) >> 23) & 0xFFu) - 127);
            uint32_t pb[NT][2];
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float c0 = row_scale[nt][0] * sc.x, c1 = row_scale[nt][1] * sc.x;
                S[nt][0] = in0 ? S[nt][0] * c0 : kNegInf;
                S[nt][1] = in0 ? S[nt][1] * c1 : kNegInf;
                S[nt][2] = in1 ? S[nt][2] * c0 : kNegInf;
                S[nt][3] = in1 ? S[nt][3] * c1 : kNegInf;
                over |= fmaxf(S[nt][0], S[nt][2]) + ev > M[nt][0] + kSlack || fmaxf(S[nt][1], S[nt][3]) + ev > M[nt][1] + kSlack;
            }
            if (__any_sync(0xffffffffu, over)) {  // raise the maximum and bring the sums to it
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(S[nt][e], S[nt][e + 2]) + ev;
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, M[nt][e]);
                        const float f = m == kNegInf ? 1.f : ex2(M[nt][e] - m);
                        M[nt][e] = m;
                        l[nt][e] *= f;
#pragma unroll
                        for (int j = 0; j < F::MT; ++j) {
                            acc[nt][j][e] *= f;
                            acc[nt][j][e + 2] *= f;
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = M[nt][0] == kNegInf ? 0.f : M[nt][0], m1 = M[nt][1] == kNegInf ? 0.f : M[nt][1];
                const float e0 = ex2(S[nt][0] - m0), e1 = ex2(S[nt][1] - m1), e2 = ex2(S[nt][2] - m0), e3 = ex2(S[nt][3] - m1);
                l[nt][0] += e0 + e2;
                l[nt][1] += e1 + e3;
                pb[nt][0] = transpose8(pack_half(e0 * sc.y, e1 * sc.y));
                pb[nt][1] = transpose8(pack_half(e2 * sc.y, e3 * sc.y));
            }
            const uint8_t *vs = slot + F::KBYTES + lane * F::VB;
            uint32_t vw[4][F::VB / 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (F::VB == 16) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(vs + i * 32 * F::VB);
                    vw[i][0] = x.x;
                    vw[i][1] = x.y;
                    vw[i][F::VB / 4 - 2] = x.z;
                    vw[i][F::VB / 4 - 1] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(vs + i * 32 * F::VB);
                    vw[i][0] = x.x;
                    vw[i][1] = x.y;
                }
            }
#pragma unroll
            for (int i = 0; i < F::VB / 4; ++i) {
                const uint32_t x = __byte_perm(vw[0][i], vw[1][i], 0x5140), y = __byte_perm(vw[0][i], vw[1][i], 0x7362);
                const uint32_t z = __byte_perm(vw[2][i], vw[3][i], 0x5140), w = __byte_perm(vw[2][i], vw[3][i], 0x7362);
                const uint32_t x0 = widen_lo(x), x1 = widen_hi(x), z0 = widen_lo(z), z1 = widen_hi(z);
                const uint32_t y0 = widen_lo(y), y1 = widen_hi(y), w0 = widen_lo(w), w1 = widen_hi(w);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_f16(acc[nt][2 * i], x0, x1, z0, z1, pb[nt][0], pb[nt][1]);
                    mma_f16(acc[nt][2 * i + 1], y0, y1, w0, w1, pb[nt][0], pb[nt][1]);
                }
            }
        }

        // ---- the warps' sums of this unit together
        __syncthreads();  // the buffer's previous use is over
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * t + e;
                float x = l[nt][e];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                if (g == 0) {
                    merge_m[warp * F::ROWS + r] = M[nt][e];
                    merge_l[warp * F::ROWS + r] = x;
                }
                float *dst = merge + (warp * F::ROWS + r) * F::PITCH + g * F::VB;
#pragma unroll
                for (int j = 0; j < F::MT; ++j)
                    *reinterpret_cast<float2 *>(dst + 2 * j) = make_float2(acc[nt][j][e], acc[nt][j][e + 2]);
            }
        __syncthreads();
        const bool whole = cur.s0 == 0 && cur.s1 == cur.steps;
        float *part = p.ws + ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * F::PART;
        for (int i = tid; i < F::ROWS * (D / 4); i += kThreads) {
            const int r = i / (D / 4), d = (i - r * (D / 4)) * 4;
            float m = kNegInf;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, merge_m[w * F::ROWS + r]);
            float sum = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = merge_m[w * F::ROWS + r], f = m == kNegInf ? 1.f : ex2(mw - m);
                const float4 x = *reinterpret_cast<const float4 *>(merge + (w * F::ROWS + r) * F::PITCH + d);
                sum += f * merge_l[w * F::ROWS + r];
                a.x += f * x.x;
                a.y += f * x.y;
                a.z += f * x.z;
                a.w += f * x.w;
            }
            if (!whole) {
                *reinterpret_cast<float4 *>(part + r * D + d) = a;
                if (d == 0) {
                    part[F::ROWS * D + r] = m;
                    part[F::ROWS * D + F::ROWS + r] = sum;
                }
            } else if (r0 + r < group) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int64_t row = (int64_t)cur.n * p.Hq + h * group + r0 + r;
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
        }
        first = false;
        left -= cur.s1 - cur.s0;
        if (left <= 0) break;
        next_segment(c, U, left, cur);
    }
    cp_wait<0>();
}

// Adds the pieces of one query row in their order along the line; a CTA for each (sequence,
// unit, row).  Rows of sequences without tokens are written here as zero.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads) attn_decode_join_kernel(const __grid_constant__ DecodeParams p, int ctas) {
    using F = Cfg<D, NT>;
    __shared__ int64_t s_scan[kWarps];
    __shared__ int64_t s_at;
    __shared__ float s_acc[kWarps][D], s_m[kWarps], s_l[kWarps];
    constexpr int C = D / 32;
    const PagedCache &c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = p.Hq / c.Hk, parts = (group + F::ROWS - 1) / F::ROWS, U = c.Hk * parts;
    const int qh = blockIdx.x, n = blockIdx.y;  // query head, sequence
    const int h = qh / group, in = qh - h * group, u = h * parts + in / F::ROWS, r = in % F::ROWS;
    const Line line = measure_line(c, s_scan);
    if (n >= line.first && n < line.last) {
        int64_t at = line.mine;
        for (int i = line.first; i < n; ++i) at += steps_of(c, i);
        s_at = at;
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = (int64_t)n * p.Hq + qh;
    const int steps = steps_of(c, n);
    float a[C] = {};
    float m = kNegInf, l = 0.f;
    if (steps > 0) {
        const int64_t S = piece_steps(line.total * U, ctas), Ls = s_at * U + (int64_t)u * steps;
        const int64_t c0 = Ls / S, c1 = (Ls + steps - 1) / S;
        if (c0 == c1) return;  // written by its CTA
        for (int64_t k = c0 + warp; k <= c1; k += kWarps) {
            // the unit is the first of its CTA's segments unless the CTA began before it
            const float *part = p.ws + (k * 2 + (k * S >= Ls ? 0 : 1)) * F::PART;
            const float mk = __ldcg(part + F::ROWS * D + r), lk = __ldcg(part + F::ROWS * D + F::ROWS + r);
            float x[C];
            if (C == 4) {
                const float4 y = __ldcg(reinterpret_cast<const float4 *>(part + r * D) + lane);
                x[0] = y.x;
                x[1] = y.y;
                x[C - 2] = y.z;
                x[C - 1] = y.w;
            } else {
                const float2 y = __ldcg(reinterpret_cast<const float2 *>(part + r * D) + lane);
                x[0] = y.x;
                x[1] = y.y;
            }
            const float mn = fmaxf(m, mk);
            const float f = mn == kNegInf ? 1.f : ex2(m - mn), fk = mn == kNegInf ? 1.f : ex2(mk - mn);
            m = mn;
            l = l * f + lk * fk;
#pragma unroll
            for (int i = 0; i < C; ++i) a[i] = a[i] * f + x[i] * fk;
        }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) s_acc[warp][lane * C + i] = a[i];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    if (tid >= D) return;
    m = kNegInf;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w]);
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = m == kNegInf ? 1.f : ex2(s_m[w] - m);
        sum += f * s_l[w];
        x += f * s_acc[w][tid];
    }
    st_out(p.o, row * D + tid, sum == 0.f ? 0.f : x / sum, p.o_bf16);
    if (p.lse && tid == 0) p.lse[row] = sum == 0.f ? kNegInf : (log2f(sum) + m) * 0.6931471805599453f;
}

int decode_ctas() { return kCtasPerSm * sm_count(); }

template <int D, int NT>
kda_status run(const DecodeParams &p, cudaStream_t st) {
    using F = Cfg<D, NT>;
    static DeviceOnce configured;
    const int dev = current_device(), ctas = decode_ctas();
    if (!configured.done(dev)) {
        if (cudaFuncSetAttribute(attn_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::SMEM) !=
            cudaSuccess) {
            set_error("attn_decode: cannot reserve shared memory: %s", cudaGetErrorString(cudaGetLastError()));
            return KDA_ERR_CUDA;
        }
        configured.set(dev);
    }
    attn_decode_kernel<D, NT><<<ctas, kThreads, F::SMEM, st>>>(p);
    note_launch();
    kda_status s = check_launch("attn_decode_kernel");
    if (s != KDA_OK) return s;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.Hq, p.c.N, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];  // starts while the first kernel ends; waits for it before it reads
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_decode_join_kernel<D, NT>, p, ctas);
    note_launch();
    if (e != cudaSuccess) {
        set_error("attn_decode_join_kernel: %s", cudaGetErrorString(e));
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return check_launch("attn_decode_join_kernel");
}

}  // namespace

size_t attn_decode_workspace_bytes(int Hq, int Hk, int D) {
    const int rows = Hq / Hk <= 8 ? 8 : 16;
    return (size_t)decode_ctas() * 2 * rows * (D + 2) * sizeof(float);
}

kda_status launch_attn_decode(const DecodeParams &p, cudaStream_t st) {
    if (p.c.N == 0) return KDA_OK;
    const bool wide = p.Hq / p.c.Hk > 8;
    if (p.c.D == 128) return wide ? run<128, 2>(p, st) : run<128, 1>(p, st);
    return wide ? run<64, 2>(p, st) : run<64, 1>(p, st);
}

}  // namespace kda
