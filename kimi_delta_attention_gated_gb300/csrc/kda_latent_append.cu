// kda_latent_append.cu -- appends tokens' latent rows to their paged cache:
//
//   [c | r]  ->  [c / sqrt(mean(c^2) + eps) * w | r turned by the token's place]
//
// in bf16, each value rounded once.  The bound is memory: 1152 bytes a token in and as many out (twice
// where the rows are wanted densely too).  A warp takes a token, a lane two 16-byte pieces of c, so that
// the norm needs no more than two warp sums, and eight lanes take the pieces of r.
#include "kda_latent.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr float kBig = 1.152921504606847e18f;     // 2^60: squares above and below these bounds
constexpr float kSmall = 8.673617379884035e-19f;  // 2^-60 leave fp32, so c is taken at another scale

// The sequence of row t: the last one that begins at or before it; -1 if t belongs to none.
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
    return t >= __ldg(p.cu_seqlens + lo) && t < __ldg(p.cu_seqlens + lo + 1) ? lo : -1;
}

__global__ void __launch_bounds__(kWarps * 32) latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
    __shared__ __align__(16) float2 s_cs[kWarps][kShared / 2];
    __shared__ __align__(16) __nv_bfloat16 s_r[kWarps][kShared];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, np = p.rot.R >> 1;
    const uint64_t turn = lane < np ? turn_of(__ldg(p.rot.inv_freq + lane)) : 0;
    float w[16];
    if (p.norm_w) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __ldg(p.norm_w + (i >> 3) * 256 + lane * 8 + (i & 7));
    }
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < p.tokens; t += (int64_t)gridDim.x * kWarps) {
        const __nv_bfloat16 *x = p.x + t * p.x_stride;
        uint4 a = __ldg(reinterpret_cast<const uint4 *>(x) + lane), b = __ldg(reinterpret_cast<const uint4 *>(x) + 32 + lane);
        uint4 r = make_uint4(0, 0, 0, 0);
        if (lane < 8) r = __ldg(reinterpret_cast<const uint4 *>(x + kLatent) + lane);
        const int n = sequence_of(p, t);
        if (n < 0) continue;  // rows of no sequence are left as they are
        const uint32_t place = (uint32_t)max(__ldg(p.c.lens + n), 0) + (p.cu_seqlens ? (uint32_t)(t - max(__ldg(p.cu_seqlens + n), 0)) : 0u);
        const uint32_t block = place >> p.c.p_shift;
        int page = -1;
        if (block < (uint32_t)p.c.max_blocks) page = __ldg(p.c.block_table + (int64_t)n * p.c.max_blocks + block);
        if (p.norm_w) {
            float v[16];
            {
                float h[8];
                Vec16<__nv_bfloat16>::load(a, h);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = h[i];
                Vec16<__nv_bfloat16>::load(b, h);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[8 + i] = h[i];
            }
            float most = 0.f, sum = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                most = fmaxf(most, fabsf(v[i]));
                sum = fmaf(v[i], v[i], sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            float s = 1.f;
            if (most > kBig || most < kSmall) {
                s = most > kBig ? exp2_int(-64) : exp2_int(64);
                if (s > 1.f && p.eps >= 0.5f) s = 1.f;  // (eps s^2 has to stay finite; such an eps is all that counts)
                sum = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) sum = fmaf(v[i] * s, v[i] * s, sum);
            }
            const float f = rsqrtf(warp_sum(sum) * (1.f / kLatent) + p.eps * s * s);
            float h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = v[i] * s * f * w[i];
            a = Vec16<__nv_bfloat16>::store(h);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = v[8 + i] * s * f * w[8 + i];
            b = Vec16<__nv_bfloat16>::store(h);
        }
        if (np > 0) {
            if (lane < 8) reinterpret_cast<uint4 *>(s_r[warp])[lane] = r;
            if (lane < np) {
                float c, s;
                cos_sin_turn((uint64_t)place * turn, c, s);
                s_cs[warp][cs_at(lane, np)] = make_float2(c, s * p.rot.sign);
            }
            __syncwarp();
            if (lane < rotary_units(kShared, p.rot.R, p.rot.interleaved, 8))
                rotate_unit<__nv_bfloat16>(s_r[warp], s_r[warp], s_cs[warp], lane, p.rot.R, p.rot.interleaved, p.rot.magnitude);
            __syncwarp();
            if (lane < 8) r = reinterpret_cast<const uint4 *>(s_r[warp])[lane];
            __syncwarp();  // read before the next token's are written
        }
        auto put = [&](__nv_bfloat16 *y) {
            uint4 *row = reinterpret_cast<uint4 *>(y);
            row[lane] = a;
            row[32 + lane] = b;
            if (lane < 8) row[64 + lane] = r;
        };
        if (p.rows_out) put(p.rows_out + t * kRow);
        if ((uint32_t)page < (uint32_t)p.c.n_pages)
            put(p.c.rows + (((int64_t)page << p.c.p_shift) + (place & (p.c.P - 1))) * kRow);
    }
}

}  // namespace

kda_status launch_latent_append(const LatentAppendParams &p, cudaStream_t st) {
    if (p.tokens == 0 || p.c.N == 0) return KDA_OK;
    const int64_t most = 8ll * sm_count(), ctas = (p.tokens + kWarps - 1) / kWarps;
    latent_append_kernel<<<(unsigned)(ctas < most ? ctas : most), kWarps * 32, 0, st>>>(p);
    note_launch();
    return check_launch("latent_append_kernel");
}

}  // namespace kda
