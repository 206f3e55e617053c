// kda_latent.cuh -- definitions shared by the latent-attention operators: the paged cache of one
// vector a token and its append (kda_latent_append.cu), the products with the projection from the
// latent to each head's keys and values (kda_latent_proj.cu), and attention over the cache
// (kda_attn_latent.cu).
//
// A token's row is [c | r]: c the 512 channels of the latent, from which every head's 128 key and
// 128 value channels are linear images, k_h = Wk_h c and v_h = Wv_h c, and r 64 key channels that
// all heads share.  A head's score of a query (qn | qr) of 128 + 64 channels is
//     qn . Wk_h c + qr . r = (Wk_h^T qn | qr) . (c | r),
// and its output sum_j p_j Wv_h c_j = Wv_h (sum_j p_j c_j): attention can run on the rows
// themselves, with queries of 576 channels and outputs of 512, as over one key head for all.
#pragma once

#include "kda_attn.cuh"

namespace kda {

constexpr int kLatent = 512;               // channels of the latent
constexpr int kShared = 64;                // key channels that the heads share
constexpr int kRow = kLatent + kShared;    // a token's row
constexpr int kHeadKey = 128, kHeadValue = 128;
constexpr int kHeadQuery = kHeadKey + kShared;

struct LatentCache {
    __nv_bfloat16 *rows;          // [pages, P, kRow]
    const int32_t *block_table;   // [N, max_blocks]
    const int32_t *lens;          // [N] tokens in the cache
    int n_pages, max_blocks, P, N;
    int p_shift;                  // P = 1 << p_shift
};

struct LatentAppendParams {
    LatentCache c;                // lens: tokens before this call
    const __nv_bfloat16 *x;       // rows of kRow, x_stride elements apart
    int64_t x_stride, tokens;
    const int32_t *cu_seqlens;    // [N + 1] or null: one token per sequence
    const float *norm_w;          // [kLatent] or null: not normalised
    float eps;
    RotaryParams rot;             // of the shared channels; R at most kShared
    __nv_bfloat16 *rows_out;      // [tokens, kRow] or null
};

enum LatentProduct { kLatentQueries = 0, kLatentValues = 1, kLatentExpand = 2 };

struct LatentProductParams {
    int what;                     // a LatentProduct
    const __nv_bfloat16 *x;       // rows x_stride elements apart
    int64_t x_stride, tokens;
    int H;
    const __nv_bfloat16 *w;       // [H, kHeadKey + kHeadValue, kLatent]
    const int32_t *positions;     // [tokens] (queries), where rot.inv_freq is given
    RotaryParams rot;
    __nv_bfloat16 *out, *out2;    // dense; expand: keys and values
    uint32_t polls;
};

struct AttnLatentParams {
    LatentCache c;                // lens: tokens to attend to, the call's own included
    const __nv_bfloat16 *q;       // rows of H * kRow, q_stride elements apart
    int64_t q_stride;
    int tokens, H;
    const int32_t *cu_seqlens;    // [N + 1] or null: one token per sequence
    float scale;
    void *o;                      // [tokens, H, kLatent]
    int o_bf16;
    float *lse;                   // [tokens, H] or null
    float *ws;                    // sums of parts of the tokens
    uint32_t polls;               // bound on the copies' waits
};

kda_status launch_latent_append(const LatentAppendParams &p, cudaStream_t st);
kda_status launch_latent_product(const LatentProductParams &p, cudaStream_t st);
size_t attn_latent_workspace_bytes(int64_t N, int64_t tokens, int H, int64_t max_tokens);
kda_status launch_attn_latent(const AttnLatentParams &p, cudaStream_t st);
int take_latent_product_timeouts(cudaStream_t st);
int take_attn_latent_timeouts(cudaStream_t st);

// Rows of sequence n in a call, clamped to the tensors.
__device__ __forceinline__ void call_rows(const int32_t *cu, int64_t tokens, int n, int64_t &t0, int &len) {
    if (!cu) {
        t0 = n;
        len = 1;
        return;
    }
    int64_t a = __ldg(cu + n), b = __ldg(cu + n + 1);
    a = max((int64_t)0, min(a, tokens));
    b = max(a, min(b, tokens));
    t0 = a;
    len = (int)(b - a);
}

// The channels 2 lane, 2 lane + 1 of r turned, from the cos and sin of pair `lane`.  Interleaved, they are that pair; else
// they belong to the pairs 2 lane and the next, whose other halves another lane has.  (By 16-byte pieces in a few lanes,
// through shared memory, 86824 tokens took 53 us instead of 39.)
__device__ __forceinline__ uint32_t turn_word(uint32_t word, float c, float s, const RotaryParams &rot) {
    const int lane = threadIdx.x & 31, np = rot.R >> 1;
    const float a = __uint_as_float(word << 16), b = __uint_as_float(word & 0xFFFF0000u);
    float x, y;
    if (rot.interleaved) {
        turn_pair(a, b, make_float2(c, s), rot.magnitude, x, y);
    } else {
        const bool first = lane < np >> 1;
        const uint32_t other = __shfl_sync(0xffffffffu, word, first ? lane + (np >> 1) : lane - (np >> 1));
        const int pair = 2 * (first ? lane : lane - (np >> 1));
        const float c0 = __shfl_sync(0xffffffffu, c, pair), s0 = __shfl_sync(0xffffffffu, s, pair);
        const float c1 = __shfl_sync(0xffffffffu, c, pair + 1), s1 = __shfl_sync(0xffffffffu, s, pair + 1);
        const uint32_t o = first ? other : other ^ 0x80008000u;  // (a' = a cos - b sin, b' = b cos + a sin)
        x = diff_of_products(a, c0, __uint_as_float(o << 16), s0) * rot.magnitude;
        y = diff_of_products(b, c1, __uint_as_float(o & 0xFFFF0000u), s1) * rot.magnitude;
    }
    return lane < np ? pack_bf16x2(x, y) : word;
}

// A launch that may set up while the one before ends: what that wrote or read is touched after before_is_over only.
template <typename... Params, typename... Args>
cudaError_t launch_beside_end(void (*kernel)(Params...), unsigned ctas, int threads, size_t smem, cudaStream_t st, const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}
inline kda_status launched(cudaError_t e, const char *what) {
    note_launch();
    if (e == cudaSuccess) return check_launch(what);
    set_error("%s: %s", what, cudaGetErrorString(e));
    cudaGetLastError();
    return KDA_ERR_CUDA;
}
__device__ __forceinline__ void before_is_over() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next launch may set up from here on.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

}  // namespace kda
