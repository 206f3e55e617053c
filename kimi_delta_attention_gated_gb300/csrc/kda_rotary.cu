// kda_rotary.cu -- rotary positions: each token's first R channels of every head, taken as
// R / 2 pairs, turned by the angle position * inv_freq[pair].
//
//   (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
//
// Memory bound: x is read once and written once.  A CTA takes a few tokens, forms their
// cos and sin once (shared by all heads) in shared memory and then turns 16-byte vectors.
// 8192 tokens of 96 heads of 128, bf16: 65.9 us, 6.1 TB/s (90 % of a copy's rate); 4099 tokens of
// 12 heads of 64, fp32, half of each turned: 6.8 us, of which the launch and one wave of CTAs take
// most; 8 tokens of 32 heads: 2.9 us, an empty launch's time.
#include "kda_attn.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kRoom = 1024;  // cos / sin pairs of a tile

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const T *x, int64_t xs, const int32_t *positions,
                                                          const RotaryParams r, T *out, int64_t os, int64_t tokens,
                                                          int H, int D, int tile) {
    __shared__ __align__(16) float2 cs[kRoom];
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int n = (int)min((int64_t)tile, tokens - t0);
    fill_cos_sin(cs, r, n, [&](int t) { return __ldg(positions + t0 + t); }, threadIdx.x, kThreads);
    __syncthreads();
    rotate_rows<T>(x + t0 * xs, xs, out + t0 * os, os, cs, r, n, H, D, threadIdx.x, kThreads);
}

}  // namespace

kda_status launch_rotary(const void *x, int bf16, int64_t x_stride, const int32_t *positions, const RotaryParams &r,
                         void *out, int64_t out_stride, int64_t T, int H, int D, cudaStream_t st) {
    if (T == 0) return KDA_OK;
    const int tile = rotary_tile_tokens(H, D, r.R, bf16 ? 8 : 4, kThreads, kRoom);
    const int64_t grid = (T + tile - 1) / tile;
    if (bf16)
        rotary_kernel<__nv_bfloat16><<<(unsigned)grid, kThreads, 0, st>>>(
            static_cast<const __nv_bfloat16 *>(x), x_stride, positions, r, static_cast<__nv_bfloat16 *>(out), out_stride,
            T, H, D, tile);
    else
        rotary_kernel<float><<<(unsigned)grid, kThreads, 0, st>>>(static_cast<const float *>(x), x_stride, positions, r,
                                                                  static_cast<float *>(out), out_stride, T, H, D, tile);
    note_launch();
    return check_launch("rotary_kernel");
}

}  // namespace kda
