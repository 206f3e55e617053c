// kda_latent_append.cu -- appends tokens' latent rows to their paged cache:
//
//   [c | r]  ->  [c / sqrt(mean(c^2) + eps) * w | r turned by the token's place]
//
// in bf16, each value rounded once.  The bound is memory: 1152 bytes a token in and as many out (twice
// where the rows are wanted densely too).  A warp takes a run of tokens, whose sequence it looks for
// once, with the next token's row on its way; a lane has two 16-byte pieces of c, so that the norm needs
// one warp sum, and two channels of r.
//
// 86824 tokens, normalised and turned, rows wanted: 53 us, 5.7 TB/s of 6.7 that a copy reaches; without the dense rows 39
// (76 %), turned or not: each warp's chain of a token, a row ahead under way.  One token of 256 sequences: 2.2 us, a launch.
#include "kda_latent.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kResident = 6;  // CTAs of an SM: 24 warps (16, 24 and 32 warps: 57.9, 52.7 and 55.0 us for 86824 tokens)
// Sums of squares within these bounds have lost nothing to fp32's range.
constexpr float kLeastSum = 8.077935669463161e-28f, kMostSum = 1.329227995784916e36f;  // 2^-90, 2^120

// The sequence of row t: the last one that begins at or before it.
__device__ __forceinline__ int sequence_of(const LatentAppendParams &p, int64_t t) {
    if (!p.cu_seqlens) return (int)t;
    int lo = 0, hi = p.c.N - 1;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (__ldg(p.cu_seqlens + m) <= t)
            lo = m;
        else
            hi = m - 1;
    }
    return lo;
}

struct Row {
    uint4 a, b;  // pieces lane and 32 + lane of c
    uint32_t r;  // channels 2 lane, 2 lane + 1 of r
};
__device__ __forceinline__ Row load_row(const LatentAppendParams &p, int64_t t) {
    const uint4 *x = reinterpret_cast<const uint4 *>(p.x + t * p.x_stride);
    const int lane = threadIdx.x & 31;
    Row y;
    y.a = __ldcs(x + lane);
    y.b = __ldcs(x + 32 + lane);
    y.r = __ldcs(reinterpret_cast<const uint32_t *>(x + 64) + lane);
    return y;
}

// c / sqrt(mean(c^2) + eps) * w.
__device__ __forceinline__ void normalise(Row &y, const float (&w)[16], float eps) {
    float v[16];
    {
        float h[8];
        Vec16<__nv_bfloat16>::load(y.a, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h[i];
        Vec16<__nv_bfloat16>::load(y.b, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 + i] = h[i];
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
    sum = warp_sum(sum);
    float s = 1.f;
    if (!(sum >= kLeastSum && sum <= kMostSum)) {  // (the same in all lanes) again at another scale
        // (512 squares of less than 2^128 s each have to stay finite, so s^2 <= 2^-138; eps s^2, too; beside an eps of 1/2 so
        // small a sum is nothing)
        s = !(sum <= kMostSum) ? exp2_int(-69) : eps < 0.5f ? exp2_int(64) : 1.f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            v[i] *= s;
            sum = fmaf(v[i], v[i], sum);
        }
        sum = warp_sum(sum);
    }
    const float f = rsqrtf(sum * (1.f / kLatent) + eps * s * s);
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = v[i] * f * w[i];
    y.a = Vec16<__nv_bfloat16>::store(h);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = v[8 + i] * f * w[8 + i];
    y.b = Vec16<__nv_bfloat16>::store(h);
}

__global__ void __launch_bounds__(kWarps * 32, kResident) latent_append_kernel(const __grid_constant__ LatentAppendParams p, int run) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, np = p.rot.R >> 1;
    const int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * run, t1 = min(t0 + run, p.tokens);
    if (t0 >= t1) return;
    before_is_over();
    Row next = load_row(p, t0);
    const uint64_t turn = lane < np ? turn_of(__ldg(p.rot.inv_freq + lane)) : 0;
    float w[16];
    if (p.norm_w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __ldg(p.norm_w + (i >> 3) * 256 + lane * 8 + (i & 7));
    }
    int n = -1;
    int64_t first = 0, end = 0;  // of sequence n
    uint32_t before = 0;         // places of it that were there
    for (int64_t t = t0; t < t1; ++t) {
        Row y = next;
        if (t + 1 < t1) next = load_row(p, t + 1);
        if (n < 0 || t >= end) {
            n = sequence_of(p, t);
            first = p.cu_seqlens ? max(__ldg(p.cu_seqlens + n), 0) : t;
            end = p.cu_seqlens ? __ldg(p.cu_seqlens + n + 1) : t + 1;
            before = (uint32_t)max(__ldg(p.c.lens + n), 0);
        }
        if (t < first || t >= end) {  // rows of no sequence are left as they are
            n = -1;
            continue;
        }
        const uint32_t place = before + (uint32_t)(t - first), block = place >> p.c.p_shift;
        int page = -1;
        if (block < (uint32_t)p.c.max_blocks) page = __ldg(p.c.block_table + (int64_t)n * p.c.max_blocks + block);
        if (p.norm_w) normalise(y, w, p.eps);
        if (np > 0) {
            float c, sn;
            cos_sin_turn((uint64_t)place * turn, c, sn);
            y.r = turn_word(y.r, c, sn, p.rot);
        }
        auto put = [&](__nv_bfloat16 *to) {
            uint4 *row = reinterpret_cast<uint4 *>(to);
            row[lane] = y.a;
            row[32 + lane] = y.b;
            reinterpret_cast<uint32_t *>(row + 64)[lane] = y.r;
        };
        if (p.rows_out) put(p.rows_out + t * kRow);
        if ((uint32_t)page < (uint32_t)p.c.n_pages)
            put(p.c.rows + (((int64_t)page << p.c.p_shift) + (place & (p.c.P - 1))) * kRow);
    }
}

}  // namespace

kda_status launch_latent_append(const LatentAppendParams &p, cudaStream_t st) {
    if (p.tokens == 0 || p.c.N == 0) return KDA_OK;
    // one token a warp, or equal runs for the warps that the GPU holds at once
    const int64_t warps = (int64_t)sm_count() * kResident * kWarps, run = (p.tokens + warps - 1) / warps;
    const int64_t ctas = (p.tokens + run * kWarps - 1) / (run * kWarps);
    const cudaError_t e = launch_beside_end(latent_append_kernel, (unsigned)ctas, kWarps * 32, 0, st, p, (int)run);
    return launched(e, "latent_append_kernel");
}

}  // namespace kda
