// kda_abi.cu -- the extern "C" boundary of libkda: argument validation, path
// selection and launch bookkeeping.  Declarations and their documentation are
// in include/kda.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "kda_attn.cuh"
#include "kda_internal.cuh"
#include "kda_latent.cuh"

namespace kda {

namespace {
thread_local char g_err[512] = "";
std::atomic<uint64_t> g_launches{0};
std::atomic<uint32_t> g_wait_polls{kDefaultWaitPolls};
constexpr int kVersion = 10300;  // 1.3.0
}  // namespace

uint32_t wait_polls() { return g_wait_polls.load(std::memory_order_relaxed); }

int current_device() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return dev;
}

void set_error(const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof(g_err), fmt, ap);
    va_end(ap);
}

void note_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

kda_status check_launch(const char *what) {
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("%s: %s", what, cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

}  // namespace kda

using kda::set_error;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Index arrays, scales and frequencies: their own size (slices of larger arrays are used as they lie).
bool aligned_to(const void *p, size_t n) { return (uintptr_t)p % n == 0; }

bool dtype_ok(int d) { return d == KDA_BF16 || d == KDA_F32; }

bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

#define KDA_REQUIRE(cond, code, ...) \
    do {                             \
        if (!(cond)) {               \
            set_error(__VA_ARGS__);  \
            return code;             \
        }                            \
    } while (0)

// A byte range of one argument, for the overlap checks.
struct Span {
    const void *p;
    size_t bytes;
    const char *name;
};

bool overlaps(const Span &a, const Span &b) {
    if (!a.p || !b.p || a.bytes == 0 || b.bytes == 0) return false;
    const char *x = static_cast<const char *>(a.p), *y = static_cast<const char *>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

// The kernels read their inputs chunk by chunk while they write their outputs, so no
// output may share bytes with an input or with another output.  The one exception is
// the state: final_state may be initial_state itself (the same pointer), never a
// partial overlap.  Returns the first offending pair in the error message.
kda_status check_overlaps(const char *fn, const Span *in, int n_in, const Span *out, int n_out, const Span &s0,
                          const Span &sT) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            KDA_REQUIRE(!overlaps(out[i], in[j]), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, out[i].name,
                        in[j].name);
        for (int j = i + 1; j < n_out; ++j)
            KDA_REQUIRE(!overlaps(out[i], out[j]), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn,
                        out[i].name, out[j].name);
        KDA_REQUIRE(!overlaps(out[i], s0) && !overlaps(out[i], sT), KDA_ERR_INVALID_ARG,
                    "%s: %s must not overlap the state", fn, out[i].name);
    }
    for (int j = 0; j < n_in; ++j)
        KDA_REQUIRE(!overlaps(sT, in[j]), KDA_ERR_INVALID_ARG, "%s: the final state must not overlap %s", fn,
                    in[j].name);
    KDA_REQUIRE(!overlaps(s0, sT) || s0.p == sT.p, KDA_ERR_INVALID_ARG,
                "%s: final_state may be initial_state itself but must not partly overlap it", fn);
    return KDA_OK;
}

size_t esize(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }

// Overlap check of one prefill / decode call: rows tokens, N sequences.
kda_status check_call_overlaps(const char *fn, const void *q, const void *k, const void *v, int qkv_dtype,
                               const void *g, size_t g_esz, const void *beta, size_t b_esz, const float *s0,
                               const float *sT, const void *o, int o_dtype, const float *states, const void *gate,
                               int gate_dtype, const float *norm_w, const void *y, int64_t rows, int N, int H, int K,
                               int V) {
    const size_t r = (size_t)rows, hk = (size_t)H * K, hv = (size_t)H * V, st = (size_t)N * H * K * V * 4;
    const Span in[] = {{q, r * hk * esize(qkv_dtype), "q"}, {k, r * hk * esize(qkv_dtype), "k"},
                       {v, r * hv * esize(qkv_dtype), "v"}, {g, r * hk * g_esz, "g"},
                       {beta, r * H * b_esz, "beta"},      {gate, gate ? r * hv * esize(gate_dtype) : 0, "gate"},
                       {norm_w, norm_w ? (size_t)V * 4 : 0, "norm_w"}};
    const Span out[] = {{o, r * hv * esize(o_dtype), "o"},
                        {y, y ? r * hv * esize(o_dtype) : 0, "y"},
                        {states, states ? r * hk * V * 4 : 0, "states"}};
    return check_overlaps(fn, in, 7, out, 3, Span{s0, s0 ? st : 0, "initial_state"},
                          Span{sT, sT ? st : 0, "final_state"});
}


// Checks shared by the prefill entry points; fills the sequence count.
kda_status check_seq_args(const char *fn, const void *q, const void *k, const void *v, int qkv_dtype,
                          const float *g, const float *beta, const float *s0, const float *sT,
                          const void *o, int o_dtype, const int32_t *cu, const int32_t *cu_host,
                          int n_seqs, int B, int T, int H, int K, int V, float scale,
                          const void *gate, int gate_dtype, const float *norm_w, float eps,
                          const void *y, int &N) {
    // with no tokens nothing is read or written but the state (empty tensors may be NULL)
    const bool no_tokens = (int64_t)B * T == 0;
    KDA_REQUIRE(no_tokens || (q && k && v && g && beta), KDA_ERR_INVALID_ARG,
                "%s: q, k, v, g and beta must not be NULL", fn);
    KDA_REQUIRE(no_tokens || o || (gate && y), KDA_ERR_INVALID_ARG,
                "%s: o may be NULL only when the gated norm writes y", fn);
    KDA_REQUIRE(dtype_ok(qkv_dtype) && dtype_ok(o_dtype) && (!gate || dtype_ok(gate_dtype)),
                KDA_ERR_UNSUPPORTED, "%s: unsupported dtype", fn);
    KDA_REQUIRE(H > 0 && T >= 0 && B > 0, KDA_ERR_INVALID_ARG, "%s: need B > 0, T >= 0, H > 0", fn);
    KDA_REQUIRE(dim_ok(K) && dim_ok(V), KDA_ERR_UNSUPPORTED, "%s: K=%d V=%d (supported: 32, 64, 128)", fn, K, V);
    KDA_REQUIRE(std::isfinite(scale), KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    KDA_REQUIRE((int64_t)B * T <= (int64_t)INT32_MAX, KDA_ERR_INVALID_ARG, "%s: B*T too large", fn);
    const void *ptrs[] = {q, k, v, g, beta, s0, sT, o, cu, gate, norm_w, y};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(!ptr || aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: every pointer must be 16-byte aligned", fn);
    if (gate) {
        KDA_REQUIRE(norm_w && (y || no_tokens), KDA_ERR_INVALID_ARG, "%s: the gated norm needs norm_w and y", fn);
        KDA_REQUIRE(eps > 0.f && std::isfinite(eps), KDA_ERR_INVALID_ARG, "%s: eps must be > 0", fn);
    }
    if (cu) {
        KDA_REQUIRE(B == 1, KDA_ERR_INVALID_ARG, "%s: varlen (cu_seqlens) needs B == 1", fn);
        KDA_REQUIRE(n_seqs > 0, KDA_ERR_INVALID_ARG, "%s: varlen needs n_seqs > 0", fn);
        if (cu_host) {
            KDA_REQUIRE(cu_host[0] == 0, KDA_ERR_INVALID_ARG, "%s: cu_seqlens[0] must be 0", fn);
            for (int i = 0; i < n_seqs; ++i)
                KDA_REQUIRE(cu_host[i + 1] >= cu_host[i], KDA_ERR_INVALID_ARG,
                            "%s: cu_seqlens must not decrease (entry %d)", fn, i + 1);
            KDA_REQUIRE(cu_host[n_seqs] == T, KDA_ERR_INVALID_ARG, "%s: cu_seqlens[n_seqs] = %d but T = %d", fn,
                        cu_host[n_seqs], T);
        }
        N = n_seqs;
    } else {
        KDA_REQUIRE(!cu_host, KDA_ERR_INVALID_ARG, "%s: cu_seqlens_host given without cu_seqlens", fn);
        N = B;
    }
    return KDA_OK;
}

kda::SeqParams make_params(const void *q, const void *k, const void *v, int qkv_dtype, const float *g,
                           const float *beta, const float *s0, float *sT, void *o, int o_dtype,
                           float *states, const int32_t *cu, int N, int T, int H, float scale,
                           int l2, const void *gate, int gate_dtype, const float *norm_w, float eps,
                           void *y) {
    kda::SeqParams p;
    p.q = q;
    p.k = k;
    p.v = v;
    p.g = g;
    p.beta = beta;
    p.s0 = s0;
    p.sT = sT;
    p.o = o;
    p.states = states;
    p.cu_seqlens = cu;
    p.cu_host = nullptr;
    p.K = 0;
    p.g_logits = nullptr;
    p.A_log = nullptr;
    p.dt_bias = nullptr;
    p.beta_logits = nullptr;
    p.g_lower = -INFINITY;
    p.g_logits_bf16 = p.beta_logits_bf16 = 0;
    p.gate = gate;
    p.norm_w = norm_w;
    p.y = y;
    p.N = N;
    p.T = T;
    p.H = H;
    p.scale = scale;
    p.eps = eps;
    p.l2norm = l2 ? 1 : 0;
    p.qkv_bf16 = qkv_dtype == KDA_BF16;
    p.o_bf16 = o_dtype == KDA_BF16;
    p.gate_bf16 = gate_dtype == KDA_BF16;
    p.polls = kda::wait_polls();
    for (int f = 0; f < 3; ++f) {
        p.cw[f] = p.cs_in[f] = nullptr;
        p.cs_out[f] = nullptr;
    }
    p.conv_w = 0;
    return p;
}

using kda::GateLogits;

kda_status check_logits(const char *fn, const GateLogits &gl, bool no_tokens) {
    KDA_REQUIRE(gl.A_log, KDA_ERR_INVALID_ARG, "%s: A_log must not be NULL", fn);
    KDA_REQUIRE(no_tokens || (gl.z && gl.b), KDA_ERR_INVALID_ARG, "%s: g_logits and beta_logits must not be NULL", fn);
    KDA_REQUIRE(dtype_ok(gl.z_dtype) && dtype_ok(gl.b_dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported logits dtype", fn);
    KDA_REQUIRE(!std::isnan(gl.lower) && gl.lower <= 0.f, KDA_ERR_INVALID_ARG,
                "%s: g_lower_bound must be <= 0 (-INFINITY for none)", fn);
    const void *ptrs[] = {gl.z, gl.A_log, gl.dt_bias, gl.b};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(!ptr || aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: every pointer must be 16-byte aligned", fn);
    return KDA_OK;
}

void set_logits(kda::SeqParams &p, const GateLogits *gl, int K) {
    p.K = K;
    p.g_logits = gl ? gl->z : nullptr;
    p.A_log = gl ? gl->A_log : nullptr;
    p.dt_bias = gl ? gl->dt_bias : nullptr;
    p.beta_logits = gl ? gl->b : nullptr;
    p.g_lower = gl ? gl->lower : -INFINITY;
    p.g_logits_bf16 = gl && gl->z_dtype == KDA_BF16;
    p.beta_logits_bf16 = gl && gl->b_dtype == KDA_BF16;
}

kda_status chunk_impl(const char *fn, const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                      const float *g, const float *beta, const GateLogits *gl, const float *initial_state,
                      float *final_state, void *o, kda_dtype o_dtype, const int32_t *cu_seqlens,
                      const int32_t *cu_seqlens_host, int n_seqs, int B, int T, int H, int K, int V, int chunk,
                      float scale, int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                      const float *norm_w, float eps, void *y, void *workspace, size_t workspace_bytes, int mode,
                      void *stream) {
    kda::g_err[0] = 0;
    int N = 0;
    // with logits, g / beta are checked through them (the recurrence never reads g / beta then)
    const float *gchk = gl ? reinterpret_cast<const float *>(gl->z) : g;
    const float *bchk = gl ? reinterpret_cast<const float *>(gl->b) : beta;
    kda_status s = check_seq_args(fn, q, k, v, qkv_dtype, gchk, bchk, initial_state, final_state, o, o_dtype,
                                  cu_seqlens, cu_seqlens_host, n_seqs, B, T, H, K, V, scale, gate, gate_dtype,
                                  norm_w, eps, y, N);
    if (s != KDA_OK) return s;
    if (gl && (s = check_logits(fn, *gl, (int64_t)B * T == 0)) != KDA_OK) return s;
    s = check_call_overlaps(fn, q, k, v, qkv_dtype, gchk, gl ? esize(gl->z_dtype) : 4, bchk,
                            gl ? esize(gl->b_dtype) : 4, initial_state, final_state, o, o_dtype, nullptr, gate,
                            gate_dtype, norm_w, y, (int64_t)B * T, N, H, K, V);
    if (s != KDA_OK) return s;
    KDA_REQUIRE(chunk == 16 || chunk == 32 || chunk == 64, KDA_ERR_UNSUPPORTED, "%s: chunk=%d (supported: 16, 32, 64)",
                fn, chunk);
    KDA_REQUIRE(mode == KDA_MODE_AUTO || mode == KDA_MODE_TENSOR || mode == KDA_MODE_FP32 || mode == KDA_MODE_SPLIT,
                KDA_ERR_INVALID_ARG, "%s: unknown mode %d", fn, mode);
    const bool tc_ok = kda::chunk_tc_supported(K, V, chunk) && qkv_dtype == KDA_BF16;
    KDA_REQUIRE((mode != KDA_MODE_TENSOR && mode != KDA_MODE_SPLIT) || tc_ok, KDA_ERR_UNSUPPORTED,
                "%s: the tensor path needs bf16 q/k/v, K = V = 128 and chunk = 64", fn);
    KDA_REQUIRE(mode != KDA_MODE_SPLIT || workspace, KDA_ERR_INVALID_ARG,
                "%s: the split form needs a workspace (kda_chunk_workspace_size)", fn);
    cudaStream_t st = (cudaStream_t)stream;
    // an empty prompt only hands the state through: the fp32 path does that without a tensor map
    const bool use_tc = tc_ok && mode != KDA_MODE_FP32 && T > 0;
    KDA_REQUIRE(!workspace || aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned",
                fn);
    if (use_tc) {
        kda::SeqParams p = make_params(q, k, v, qkv_dtype, g, beta, initial_state, final_state, o, o_dtype, nullptr,
                                       cu_seqlens, N, T, H, scale, use_qk_l2norm, gate, gate_dtype, norm_w, eps, y);
        p.cu_host = cu_seqlens_host;
        set_logits(p, gl, K);
        if (!workspace) return kda::launch_chunk_tc(p, K, V, chunk, st);
        const int64_t rows = (int64_t)B * T;
        const size_t need = kda::chunk_workspace_bytes(rows, N, H);
        KDA_REQUIRE(workspace_bytes >= need, KDA_ERR_INVALID_ARG,
                    "%s: the workspace holds %zu bytes, this call needs %zu (kda_chunk_workspace_size)", fn,
                    workspace_bytes, need);
        {  // the workspace is written while every tensor of the call is in use
            const size_t r = (size_t)rows, qkv = esize(qkv_dtype), st_bytes = (size_t)N * H * K * V * 4;
            const Span ws{workspace, need, "the workspace"};
            const Span all[] = {{q, r * H * K * qkv, "q"}, {k, r * H * K * qkv, "k"}, {v, r * H * V * qkv, "v"},
                                {gchk, r * H * K * (gl ? esize(gl->z_dtype) : 4), "g"},
                                {bchk, r * H * (gl ? esize(gl->b_dtype) : 4), "beta"},
                                {o, o ? r * H * V * esize(o_dtype) : 0, "o"},
                                {y, y ? r * H * V * esize(o_dtype) : 0, "y"},
                                {gate, gate ? r * H * V * esize(gate_dtype) : 0, "gate"},
                                {initial_state, initial_state ? st_bytes : 0, "initial_state"},
                                {final_state, final_state ? st_bytes : 0, "final_state"}};
            for (const Span &x : all)
                KDA_REQUIRE(!overlaps(ws, x), KDA_ERR_INVALID_ARG, "%s: the workspace must not overlap %s", fn, x.name);
        }
        if (mode != KDA_MODE_SPLIT) return kda::launch_chunk_concurrent(p, workspace, st);
        s = kda::launch_chunk_prep(p, workspace, st);
        if (s != KDA_OK) return s;
        return kda::launch_chunk_chain(p, workspace, st);
    }
    // fp32 path: o goes to y's buffer when o is not wanted, then the norm runs in place.
    void *o_target = o ? o : y;
    kda::SeqParams p = make_params(q, k, v, qkv_dtype, g, beta, initial_state, final_state, o_target, o_dtype,
                                   nullptr, cu_seqlens, N, T, H, scale, use_qk_l2norm, nullptr, gate_dtype, norm_w,
                                   eps, nullptr);
    set_logits(p, gl, K);
    s = kda::launch_chunk_fp32(p, K, V, chunk, nullptr, st);
    if (s != KDA_OK || !gate || (int64_t)B * T == 0) return s;
    return kda::launch_gated_rmsnorm(o_target, o_dtype == KDA_BF16, gate, gate_dtype == KDA_BF16, norm_w, eps, y,
                                     o_dtype == KDA_BF16, (int64_t)B * T, H, V, st);
}

// The fused short convolutions of kda_recurrent_step_conv.
struct ConvArgs {
    const float *const *w;       // [3]
    int W;
    const float *const *s_in;    // [3] or null
    float *const *s_out;         // [3]
};

// Arguments of the fused convolutions: shapes, alignment, and that no new history
// overlaps anything but its own old history (then exactly), and no weight or old history
// overlaps an output of the step.
kda_status check_conv(const char *fn, const ConvArgs &cv, int B, int H, int K, int V, const Span *step_in, int n_in,
                      const Span *step_out, int n_out) {
    KDA_REQUIRE(K == 128 && V == 128, KDA_ERR_UNSUPPORTED,
                "%s: the fused short convolutions are built for K = V = 128 (got K=%d V=%d)", fn, K, V);
    KDA_REQUIRE(cv.W >= 2 && cv.W <= 4, KDA_ERR_UNSUPPORTED, "%s: W=%d (supported: 2, 3, 4)", fn, cv.W);
    KDA_REQUIRE(cv.w && cv.s_out, KDA_ERR_INVALID_ARG, "%s: conv_weight and conv_state_out must not be NULL", fn);
    const bool hist = cv.s_in && cv.s_in[0];
    for (int f = 0; f < 3; ++f) {
        KDA_REQUIRE(cv.w[f] && cv.s_out[f], KDA_ERR_INVALID_ARG,
                    "%s: all three conv_weight and conv_state_out pointers are needed", fn);
        KDA_REQUIRE(!cv.s_in || (cv.s_in[f] != nullptr) == hist, KDA_ERR_INVALID_ARG,
                    "%s: conv_state_in gives all three histories or none", fn);
        KDA_REQUIRE(aligned16(cv.w[f]) && aligned16(cv.s_out[f]) && (!hist || aligned16(cv.s_in[f])),
                    KDA_ERR_INVALID_ARG, "%s: every pointer must be 16-byte aligned", fn);
    }
    const size_t D = (size_t)H * 128, wb = D * cv.W * 4, sb = (size_t)B * (cv.W - 1) * D * 4;
    const char *names_w[3] = {"conv_weight[0]", "conv_weight[1]", "conv_weight[2]"};
    const char *names_i[3] = {"conv_state_in[0]", "conv_state_in[1]", "conv_state_in[2]"};
    const char *names_o[3] = {"conv_state_out[0]", "conv_state_out[1]", "conv_state_out[2]"};
    for (int f = 0; f < 3; ++f) {
        const Span so{cv.s_out[f], sb, names_o[f]};
        for (int j = 0; j < n_in; ++j)
            KDA_REQUIRE(!overlaps(so, step_in[j]), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, so.name,
                        step_in[j].name);
        for (int j = 0; j < n_out; ++j)
            KDA_REQUIRE(!overlaps(so, step_out[j]), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, so.name,
                        step_out[j].name);
        for (int e = 0; e < 3; ++e) {
            const Span we{cv.w[e], wb, names_w[e]};
            KDA_REQUIRE(!overlaps(so, we), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, so.name, we.name);
            if (hist) {
                const Span si{cv.s_in[e], sb, names_i[e]};
                KDA_REQUIRE(!overlaps(so, si) || (e == f && si.p == so.p), KDA_ERR_INVALID_ARG,
                            "%s: %s may be %s itself but must not overlap any other history", fn, so.name,
                            names_i[f]);
            }
            if (e > f) {
                const Span so2{cv.s_out[e], sb, names_o[e]};
                KDA_REQUIRE(!overlaps(so, so2), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, so.name,
                            so2.name);
            }
        }
        // the weights and old histories are inputs: no output of the step may overlap them
        const Span we{cv.w[f], wb, names_w[f]}, si{hist ? cv.s_in[f] : nullptr, sb, names_i[f]};
        for (int j = 0; j < n_out; ++j)
            KDA_REQUIRE(!overlaps(we, step_out[j]) && !overlaps(si, step_out[j]), KDA_ERR_INVALID_ARG,
                        "%s: %s must not overlap %s or %s", fn, step_out[j].name, we.name, si.name);
    }
    return KDA_OK;
}

kda_status step_impl(const char *fn, const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                     const float *g, const float *beta, const GateLogits *gl, const float *state_in,
                     float *state_out, void *o, kda_dtype o_dtype, int B, int H, int K, int V, float scale,
                     int use_qk_l2norm, const void *gate, kda_dtype gate_dtype, const float *norm_w, float eps,
                     void *y, void *stream, const ConvArgs *cv = nullptr) {
    kda::g_err[0] = 0;
    int N = 0;
    KDA_REQUIRE(state_out, KDA_ERR_INVALID_ARG, "%s: state_out must not be NULL", fn);
    const float *gchk = gl ? reinterpret_cast<const float *>(gl->z) : g;
    const float *bchk = gl ? reinterpret_cast<const float *>(gl->b) : beta;
    kda_status s = check_seq_args(fn, q, k, v, qkv_dtype, gchk, bchk, state_in, state_out, o, o_dtype, nullptr,
                                  nullptr, 0, B, 1, H, K, V, scale, gate, gate_dtype, norm_w, eps, y, N);
    if (s != KDA_OK) return s;
    if (gl && (s = check_logits(fn, *gl, false)) != KDA_OK) return s;
    s = check_call_overlaps(fn, q, k, v, qkv_dtype, gchk, gl ? esize(gl->z_dtype) : 4, bchk,
                            gl ? esize(gl->b_dtype) : 4, state_in, state_out, o, o_dtype, nullptr, gate, gate_dtype,
                            norm_w, y, B, N, H, K, V);
    if (s != KDA_OK) return s;
    if (cv) {
        const size_t hk = (size_t)B * H * K, hv = (size_t)B * H * V, st = (size_t)B * H * K * V * 4;
        const Span in[] = {{q, hk * esize(qkv_dtype), "q"},
                           {k, hk * esize(qkv_dtype), "k"},
                           {v, hv * esize(qkv_dtype), "v"},
                           {gchk, hk * (gl ? esize(gl->z_dtype) : 4), gl ? "g_logits" : "g"},
                           {bchk, (size_t)B * H * (gl ? esize(gl->b_dtype) : 4), gl ? "beta_logits" : "beta"},
                           {gate, gate ? hv * esize(gate_dtype) : 0, "gate"},
                           {norm_w, norm_w ? (size_t)V * 4 : 0, "norm_w"},
                           {state_in, state_in ? st : 0, "state_in"}};
        const Span out[] = {{o, o ? hv * esize(o_dtype) : 0, "o"},
                            {y, y ? hv * esize(o_dtype) : 0, "y"},
                            {state_out, st, "state_out"}};
        if ((s = check_conv(fn, *cv, B, H, K, V, in, 8, out, 3)) != KDA_OK) return s;
    }
    kda::SeqParams p = make_params(q, k, v, qkv_dtype, g, beta, state_in, state_out, o, o_dtype, nullptr, nullptr, N,
                                   1, H, scale, use_qk_l2norm, gate, gate_dtype, norm_w, eps, y);
    set_logits(p, gl, K);
    if (cv) {
        const bool hist = cv->s_in && cv->s_in[0];
        for (int f = 0; f < 3; ++f) {
            p.cw[f] = cv->w[f];
            p.cs_in[f] = hist ? cv->s_in[f] : nullptr;
            p.cs_out[f] = cv->s_out[f];
        }
        p.conv_w = cv->W;
    }
    return kda::launch_recurrent(p, K, V, (cudaStream_t)stream);
}

// ---------------------------------------------------------------------------
// full attention

// A tensor of `rows` rows of `row` elements, `stride` elements apart.
size_t strided_bytes(int64_t rows, int64_t row, int64_t stride, size_t esz) {
    return rows == 0 ? 0 : ((size_t)(rows - 1) * stride + row) * esz;
}

kda_status check_stride(const char *fn, const char *name, int64_t stride, int64_t row, size_t esz) {
    KDA_REQUIRE(stride >= row && stride * (int64_t)esz % 16 == 0, KDA_ERR_INVALID_ARG,
                "%s: the stride of %s must be at least a row and a multiple of 16 bytes (got %lld elements)", fn, name,
                (long long)stride);
    return KDA_OK;
}

kda_status check_rotary_args(const char *fn, const double *inv_freq, float magnitude, int R, int layout, int dim) {
    KDA_REQUIRE(layout == KDA_ROTARY_HALF || layout == KDA_ROTARY_INTERLEAVED, KDA_ERR_INVALID_ARG,
                "%s: unknown rotary layout %d", fn, layout);
    KDA_REQUIRE(R >= 0 && R <= dim, KDA_ERR_INVALID_ARG, "%s: rotary_dim=%d must lie in [0, dim]", fn, R);
    KDA_REQUIRE(R % 16 == 0, KDA_ERR_UNSUPPORTED, "%s: rotary_dim=%d must be a multiple of 16", fn, R);
    KDA_REQUIRE((R > 0) == (inv_freq != nullptr), KDA_ERR_INVALID_ARG,
                "%s: inv_freq and rotary_dim > 0 come together", fn);
    KDA_REQUIRE(std::isfinite(magnitude), KDA_ERR_INVALID_ARG, "%s: magnitude must be finite", fn);
    KDA_REQUIRE(aligned_to(inv_freq, 8), KDA_ERR_INVALID_ARG, "%s: inv_freq must be 8-byte aligned", fn);
    return KDA_OK;
}

kda_status check_cache_args(const char *fn, const void *k, const void *v, const float *ks, const float *vs,
                            int num_pages, int page_size, const int32_t *table, int max_blocks, const int32_t *lens,
                            int n_seqs, int q_heads, int kv_heads, int dim) {
    KDA_REQUIRE(kv_heads > 0 && q_heads >= 0 && dim > 0 && n_seqs >= 0 && num_pages > 0 && max_blocks > 0,
                KDA_ERR_INVALID_ARG, "%s: need positive heads, dim, num_pages and max_blocks", fn);
    KDA_REQUIRE(dim == 64 || dim == 128, KDA_ERR_UNSUPPORTED, "%s: dim=%d (supported: 64, 128)", fn, dim);
    KDA_REQUIRE(page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128, KDA_ERR_UNSUPPORTED,
                "%s: page_size=%d (supported: 16, 32, 64, 128)", fn, page_size);
    KDA_REQUIRE(k && v && ks && vs, KDA_ERR_INVALID_ARG, "%s: the cache and its scales must not be NULL", fn);
    KDA_REQUIRE(n_seqs == 0 || (table && lens), KDA_ERR_INVALID_ARG,
                "%s: block_table and the lengths must not be NULL", fn);
    KDA_REQUIRE(q_heads % kv_heads == 0, KDA_ERR_INVALID_ARG, "%s: q_heads=%d is not a multiple of kv_heads=%d", fn,
                q_heads, kv_heads);
    KDA_REQUIRE(n_seqs <= 65535 && kv_heads <= 65535 && q_heads <= (1 << 20), KDA_ERR_UNSUPPORTED,
                "%s: at most 65535 sequences and heads", fn);
    KDA_REQUIRE((int64_t)num_pages * kv_heads * page_size <= INT32_MAX - 256, KDA_ERR_UNSUPPORTED,
                "%s: num_pages * kv_heads * page_size must stay below 2^31 - 256", fn);
    KDA_REQUIRE((int64_t)max_blocks * page_size <= INT32_MAX - 256, KDA_ERR_INVALID_ARG,
                "%s: max_blocks * page_size must stay below 2^31 - 256", fn);
    KDA_REQUIRE(aligned16(k) && aligned16(v), KDA_ERR_INVALID_ARG, "%s: the cache must be 16-byte aligned", fn);
    const void *words[] = {ks, vs, table, lens};
    for (const void *ptr : words)
        KDA_REQUIRE(aligned_to(ptr, 4), KDA_ERR_INVALID_ARG, "%s: scales, block_table and lengths must be 4-byte aligned",
                    fn);
    return KDA_OK;
}

// The paged cache of latent rows and what says where a sequence's tokens lie in it.
kda_status check_latent_cache(const char *fn, const void *cache, int num_pages, int page_size, const int32_t *table,
                              int max_blocks, const int32_t *lens, const int32_t *cu, int n_seqs, int64_t tokens) {
    KDA_REQUIRE(num_pages > 0 && max_blocks > 0 && n_seqs >= 0 && tokens >= 0, KDA_ERR_INVALID_ARG,
                "%s: need positive num_pages and max_blocks, n_seqs >= 0 and tokens >= 0", fn);
    KDA_REQUIRE(page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128, KDA_ERR_UNSUPPORTED,
                "%s: page_size=%d (supported: 16, 32, 64, 128)", fn, page_size);
    KDA_REQUIRE(cache, KDA_ERR_INVALID_ARG, "%s: the cache must not be NULL", fn);
    KDA_REQUIRE(n_seqs == 0 || (table && lens), KDA_ERR_INVALID_ARG, "%s: block_table and the lengths must not be NULL", fn);
    KDA_REQUIRE(tokens == 0 || n_seqs > 0, KDA_ERR_INVALID_ARG, "%s: tokens without sequences", fn);
    KDA_REQUIRE(cu || tokens == n_seqs, KDA_ERR_INVALID_ARG,
                "%s: without cu_seqlens there is one token per sequence (tokens=%lld, n_seqs=%d)", fn, (long long)tokens, n_seqs);
    KDA_REQUIRE(n_seqs <= 65535 && tokens <= (1 << 30), KDA_ERR_UNSUPPORTED, "%s: at most 65535 sequences and 2^30 tokens", fn);
    KDA_REQUIRE((int64_t)num_pages * page_size <= INT32_MAX - 256, KDA_ERR_UNSUPPORTED,
                "%s: num_pages * page_size must stay below 2^31 - 256", fn);
    KDA_REQUIRE((int64_t)max_blocks * page_size <= INT32_MAX - 256, KDA_ERR_INVALID_ARG,
                "%s: max_blocks * page_size must stay below 2^31 - 256", fn);
    KDA_REQUIRE(aligned16(cache), KDA_ERR_INVALID_ARG, "%s: the cache must be 16-byte aligned", fn);
    const void *words[] = {table, lens, cu};
    for (const void *ptr : words)
        KDA_REQUIRE(aligned_to(ptr, 4), KDA_ERR_INVALID_ARG, "%s: block_table, lengths and cu_seqlens must be 4-byte aligned", fn);
    return KDA_OK;
}

// Arguments of the products with the projection from the latent: rows of `row` elements.
kda_status check_latent_product(const char *fn, const void *x, const char *x_name, int64_t stride, int64_t row, int64_t tokens,
                                int heads, const void *w, const void *out, const void *out2) {
    KDA_REQUIRE(tokens >= 0 && heads > 0, KDA_ERR_INVALID_ARG, "%s: need tokens >= 0 and heads > 0", fn);
    KDA_REQUIRE(tokens <= (1 << 30) && heads <= 4096 && (tokens + 127) / 128 * heads <= INT32_MAX / 8, KDA_ERR_UNSUPPORTED,
                "%s: at most 4096 heads, 2^30 tokens and 2^28 tiles of 128 tokens of a head", fn);
    KDA_REQUIRE(w && (tokens == 0 || (x && out && out2)), KDA_ERR_INVALID_ARG, "%s: no tensor may be NULL", fn);
    const void *ptrs[] = {x, w, out, out2};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: every tensor must be 16-byte aligned", fn);
    return check_stride(fn, x_name, stride, row, 2);
}

// No output shares bytes with an input or with another output.
kda_status check_apart(const char *fn, const Span *in, int n_in, const Span *out, int n_out) {
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            KDA_REQUIRE(!overlaps(out[i], in[j]), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn, out[i].name,
                        in[j].name);
        for (int j = i + 1; j < n_out; ++j)
            KDA_REQUIRE(!overlaps(out[i], out[j]), KDA_ERR_INVALID_ARG, "%s: %s must not overlap %s", fn,
                        out[i].name, out[j].name);
    }
    return KDA_OK;
}

}  // namespace

namespace kda {

kda_status chunk_fwd_entry(const char *fn, const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                           const float *g, const float *beta, const float *initial_state, float *final_state, void *o,
                           kda_dtype o_dtype, const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int n_seqs,
                           int B, int T, int H, int K, int V, int chunk, float scale, int use_qk_l2norm,
                           const void *gate, kda_dtype gate_dtype, const float *norm_w, float eps, void *y,
                           void *workspace, size_t workspace_bytes, int mode, void *stream) {
    return chunk_impl(fn, q, k, v, qkv_dtype, g, beta, nullptr, initial_state, final_state, o, o_dtype, cu_seqlens,
                      cu_seqlens_host, n_seqs, B, T, H, K, V, chunk, scale, use_qk_l2norm, gate, gate_dtype, norm_w,
                      eps, y, workspace, workspace_bytes, mode, stream);
}

kda_status chunk_call(const char *fn, const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                      const float *g, const float *beta, const GateLogits *gl, const float *initial_state,
                      float *final_state, void *o, kda_dtype o_dtype, int B, int T, int H, int K, int V, int chunk,
                      float scale, int use_qk_l2norm, const void *gate, kda_dtype gate_dtype, const float *norm_w,
                      float eps, void *y, int mode, void *stream) {
    return chunk_impl(fn, q, k, v, qkv_dtype, g, beta, gl, initial_state, final_state, o, o_dtype, nullptr, nullptr,
                      0, B, T, H, K, V, chunk, scale, use_qk_l2norm, gate, gate_dtype, norm_w, eps, y, nullptr, 0,
                      mode, stream);
}

}  // namespace kda

extern "C" {

int kda_version(void) { return kda::kVersion; }

const char *kda_last_error(void) { return kda::g_err; }

const char *kda_status_string(int s) {
    switch (s) {
        case KDA_OK: return "KDA_OK";
        case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG";
        case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
        case KDA_ERR_CUDA: return "KDA_ERR_CUDA";
        case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT";
        default: return "KDA_ERR_UNKNOWN";
    }
}

uint64_t kda_launch_count(void) { return kda::g_launches.load(std::memory_order_relaxed); }

kda_status kda_device_status(void *stream) {
    kda::g_err[0] = 0;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) {
        set_error("kda_device_status: the stream failed: %s", cudaGetErrorString(e));
        return KDA_ERR_CUDA;
    }
    const int n_tc0 = kda::take_chunk_tc_timeouts(st);
    const int n_prep = kda::take_chunk_prep_timeouts(st);
    const int n_chain = kda::take_chunk_chain_timeouts(st);
    const int n_dec = kda::take_decode_timeouts(st);
    const int n_conv = kda::take_short_conv_timeouts(st);
    const int n_proj = kda::take_oproj_timeouts(st);
    const int n_attn_p = kda::take_attn_prompt_timeouts(st), n_attn_d = kda::take_attn_decode_timeouts(st);
    const int n_attn_l = kda::take_attn_latent_timeouts(st), n_lat = kda::take_latent_product_timeouts(st);
    if (n_tc0 < 0 || n_prep < 0 || n_chain < 0 || n_dec < 0 || n_conv < 0 || n_proj < 0 || n_attn_p < 0 || n_attn_d < 0 ||
        n_attn_l < 0 || n_lat < 0)
        return KDA_ERR_CUDA;
    const int n_attn = n_attn_p + n_attn_d + n_attn_l;
    const int n_tc = n_tc0 + n_prep + n_chain;
    if (n_tc + n_dec + n_conv + n_proj + n_attn + n_lat > 0) {
        set_error("kda_device_status: bounded waits gave up in %d prefill, %d decode, %d short-convolution, %d "
                  "output-projection, %d attention and %d latent-product CTAs; their outputs hold NaN",
                  n_tc, n_dec, n_conv, n_proj, n_attn, n_lat);
        return KDA_ERR_TIMEOUT;
    }
    return KDA_OK;
}

kda_status kda_chunk_prepass_hits(void *stream, uint64_t *chunks) {
    kda::g_err[0] = 0;
    KDA_REQUIRE(chunks, KDA_ERR_INVALID_ARG, "kda_chunk_prepass_hits: chunks must not be NULL");
    const long long n = kda::take_chunk_blob_chunks((cudaStream_t)stream);
    if (n < 0) return KDA_ERR_CUDA;
    *chunks = (uint64_t)n;
    return KDA_OK;
}

kda_status kda_set_wait_limit(int64_t polls) {
    kda::g_err[0] = 0;
    KDA_REQUIRE(polls <= (int64_t)UINT32_MAX, KDA_ERR_INVALID_ARG, "kda_set_wait_limit: at most %u polls",
                UINT32_MAX);
    kda::g_wait_polls.store(polls < 0 ? kda::kDefaultWaitPolls : (uint32_t)polls, std::memory_order_relaxed);
    return KDA_OK;
}

kda_status kda_chunk_fwd(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                         const float *g, const float *beta, const float *initial_state,
                         float *final_state, void *o, kda_dtype o_dtype,
                         const int32_t *cu_seqlens, const int32_t *cu_seqlens_host, int n_seqs,
                         int B, int T, int H, int K, int V, int chunk, float scale,
                         int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                         const float *norm_w, float eps, void *y, void *workspace, size_t workspace_bytes, int mode,
                         void *stream) {
    return chunk_impl("kda_chunk_fwd", q, k, v, qkv_dtype, g, beta, nullptr, initial_state, final_state, o, o_dtype,
                      cu_seqlens, cu_seqlens_host, n_seqs, B, T, H, K, V, chunk, scale, use_qk_l2norm, gate,
                      gate_dtype, norm_w, eps, y, workspace, workspace_bytes, mode, stream);
}

size_t kda_chunk_workspace_size(int B, int T, int H, int n_seqs) {
    if (B <= 0 || T < 0 || H <= 0 || n_seqs < 0) return 0;
    const int N = n_seqs > 0 ? n_seqs : B;
    return kda::chunk_workspace_bytes((int64_t)B * T, N, H);
}

kda_status kda_chunk_fwd_logits(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                kda_dtype beta_logits_dtype, const float *initial_state, float *final_state,
                                void *o, kda_dtype o_dtype, const int32_t *cu_seqlens,
                                const int32_t *cu_seqlens_host, int n_seqs, int B, int T, int H, int K, int V,
                                int chunk, float scale, int use_qk_l2norm, const void *gate,
                                kda_dtype gate_dtype, const float *norm_w, float eps, void *y, void *workspace,
                                size_t workspace_bytes, int mode, void *stream) {
    const GateLogits gl{g_logits, g_logits_dtype, A_log, dt_bias, g_lower_bound, beta_logits, beta_logits_dtype};
    return chunk_impl("kda_chunk_fwd_logits", q, k, v, qkv_dtype, nullptr, nullptr, &gl, initial_state, final_state,
                      o, o_dtype, cu_seqlens, cu_seqlens_host, n_seqs, B, T, H, K, V, chunk, scale, use_qk_l2norm,
                      gate, gate_dtype, norm_w, eps, y, workspace, workspace_bytes, mode, stream);
}

kda_status kda_recurrent_fwd(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                             const float *g, const float *beta, const float *initial_state,
                             float *final_state, void *o, kda_dtype o_dtype, float *states,
                             const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                             int n_seqs, int B, int T, int H, int K, int V, float scale,
                             int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                             const float *norm_w, float eps, void *y, void *stream) {
    kda::g_err[0] = 0;
    int N = 0;
    kda_status s = check_seq_args("kda_recurrent_fwd", q, k, v, qkv_dtype, g, beta, initial_state,
                                  final_state, o, o_dtype, cu_seqlens, cu_seqlens_host, n_seqs, B, T,
                                  H, K, V, scale, gate, gate_dtype, norm_w, eps, y, N);
    if (s != KDA_OK) return s;
    KDA_REQUIRE(!states || aligned16(states), KDA_ERR_INVALID_ARG, "kda_recurrent_fwd: states must be 16-byte aligned");
    s = check_call_overlaps("kda_recurrent_fwd", q, k, v, qkv_dtype, g, 4, beta, 4, initial_state, final_state, o,
                            o_dtype, states, gate, gate_dtype, norm_w, y, (int64_t)B * T, N, H, K, V);
    if (s != KDA_OK) return s;
    kda::SeqParams p = make_params(q, k, v, qkv_dtype, g, beta, initial_state, final_state, o, o_dtype,
                                   states, cu_seqlens, N, T, H, scale, use_qk_l2norm, gate, gate_dtype,
                                   norm_w, eps, y);
    set_logits(p, nullptr, K);
    return kda::launch_recurrent(p, K, V, (cudaStream_t)stream);
}

kda_status kda_recurrent_step(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                              const float *g, const float *beta, const float *state_in,
                              float *state_out, void *o, kda_dtype o_dtype, int B, int H, int K,
                              int V, float scale, int use_qk_l2norm, const void *gate,
                              kda_dtype gate_dtype, const float *norm_w, float eps, void *y,
                              void *stream) {
    return step_impl("kda_recurrent_step", q, k, v, qkv_dtype, g, beta, nullptr, state_in, state_out, o, o_dtype, B,
                     H, K, V, scale, use_qk_l2norm, gate, gate_dtype, norm_w, eps, y, stream);
}

kda_status kda_recurrent_step_logits(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                     const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                     const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                     kda_dtype beta_logits_dtype, const float *state_in, float *state_out,
                                     void *o, kda_dtype o_dtype, int B, int H, int K, int V, float scale,
                                     int use_qk_l2norm, const void *gate, kda_dtype gate_dtype,
                                     const float *norm_w, float eps, void *y, void *stream) {
    const GateLogits gl{g_logits, g_logits_dtype, A_log, dt_bias, g_lower_bound, beta_logits, beta_logits_dtype};
    return step_impl("kda_recurrent_step_logits", q, k, v, qkv_dtype, nullptr, nullptr, &gl, state_in, state_out, o,
                     o_dtype, B, H, K, V, scale, use_qk_l2norm, gate, gate_dtype, norm_w, eps, y, stream);
}

kda_status kda_recurrent_step_conv(const void *q, const void *k, const void *v, kda_dtype qkv_dtype,
                                   const float *const conv_weight[3], int W, const float *const conv_state_in[3],
                                   float *const conv_state_out[3], const float *g, const float *beta,
                                   const void *g_logits, kda_dtype g_logits_dtype, const float *A_log,
                                   const float *dt_bias, float g_lower_bound, const void *beta_logits,
                                   kda_dtype beta_logits_dtype, const float *state_in, float *state_out, void *o,
                                   kda_dtype o_dtype, int B, int H, int K, int V, float scale, int use_qk_l2norm,
                                   const void *gate, kda_dtype gate_dtype, const float *norm_w, float eps, void *y,
                                   void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_recurrent_step_conv";
    const bool plain = g || beta, logits = g_logits || beta_logits || A_log;
    KDA_REQUIRE(plain != logits, KDA_ERR_INVALID_ARG,
                "%s: give either g and beta or g_logits, A_log and beta_logits, not both or neither", fn);
    const ConvArgs cv{conv_weight, W, conv_state_in, conv_state_out};
    if (logits) {
        const GateLogits gl{g_logits, g_logits_dtype, A_log, dt_bias, g_lower_bound, beta_logits, beta_logits_dtype};
        return step_impl(fn, q, k, v, qkv_dtype, nullptr, nullptr, &gl, state_in, state_out, o, o_dtype, B, H, K, V,
                         scale, use_qk_l2norm, gate, gate_dtype, norm_w, eps, y, stream, &cv);
    }
    return step_impl(fn, q, k, v, qkv_dtype, g, beta, nullptr, state_in, state_out, o, o_dtype, B, H, K, V, scale,
                     use_qk_l2norm, gate, gate_dtype, norm_w, eps, y, stream, &cv);
}

kda_status kda_gated_rmsnorm(const void *o, kda_dtype o_dtype, const void *gate,
                             kda_dtype gate_dtype, const float *w, float eps, void *y,
                             kda_dtype y_dtype, int64_t rows, int H, int V, void *stream) {
    kda::g_err[0] = 0;
    KDA_REQUIRE((o && gate && y) || rows == 0, KDA_ERR_INVALID_ARG,
                "kda_gated_rmsnorm: o, gate and y must not be NULL");
    KDA_REQUIRE(w, KDA_ERR_INVALID_ARG, "kda_gated_rmsnorm: w must not be NULL");
    KDA_REQUIRE(dtype_ok(o_dtype) && dtype_ok(gate_dtype) && dtype_ok(y_dtype), KDA_ERR_UNSUPPORTED,
                "kda_gated_rmsnorm: unsupported dtype");
    KDA_REQUIRE(rows >= 0 && H > 0, KDA_ERR_INVALID_ARG, "kda_gated_rmsnorm: need rows >= 0 and H > 0");
    KDA_REQUIRE(dim_ok(V), KDA_ERR_UNSUPPORTED, "kda_gated_rmsnorm: V=%d (supported: 32, 64, 128)", V);
    KDA_REQUIRE(eps > 0.f && std::isfinite(eps), KDA_ERR_INVALID_ARG, "kda_gated_rmsnorm: eps must be > 0");
    KDA_REQUIRE(aligned16(o) && aligned16(gate) && aligned16(w) && aligned16(y), KDA_ERR_INVALID_ARG,
                "kda_gated_rmsnorm: every pointer must be 16-byte aligned");
    KDA_REQUIRE(o != y || o_dtype == y_dtype, KDA_ERR_INVALID_ARG,
                "kda_gated_rmsnorm: in place (o == y) needs o_dtype == y_dtype");
    return kda::launch_gated_rmsnorm(o, o_dtype == KDA_BF16, gate, gate_dtype == KDA_BF16, w, eps, y,
                                     y_dtype == KDA_BF16, rows, H, V, (cudaStream_t)stream);
}

kda_status kda_short_conv_fwd(const void *x, kda_dtype x_dtype, const float *weight, const float *bias,
                              const float *conv_state_in, float *conv_state_out, void *y,
                              kda_dtype y_dtype, const int32_t *cu_seqlens,
                              const int32_t *cu_seqlens_host, int n_seqs, int B, int T, int D, int W,
                              int activation, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_short_conv_fwd";
    const int64_t rows = (int64_t)B * T;
    KDA_REQUIRE(B > 0 && T >= 0 && D > 0, KDA_ERR_INVALID_ARG, "%s: need B > 0, T >= 0, D > 0", fn);
    KDA_REQUIRE(rows == 0 || (x && y), KDA_ERR_INVALID_ARG, "%s: x and y must not be NULL", fn);
    KDA_REQUIRE(weight, KDA_ERR_INVALID_ARG, "%s: weight must not be NULL", fn);
    KDA_REQUIRE(dtype_ok(x_dtype) && dtype_ok(y_dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported dtype", fn);
    KDA_REQUIRE(W >= 2 && W <= 4, KDA_ERR_UNSUPPORTED, "%s: W=%d (supported: 2, 3, 4)", fn, W);
    KDA_REQUIRE(D % 8 == 0, KDA_ERR_UNSUPPORTED, "%s: D=%d must be a multiple of 8", fn, D);
    KDA_REQUIRE(activation == 0 || activation == 1, KDA_ERR_INVALID_ARG, "%s: activation must be 0 or 1", fn);
    KDA_REQUIRE(rows <= (int64_t)INT32_MAX, KDA_ERR_INVALID_ARG, "%s: B*T=%lld too large", fn, (long long)rows);
    const void *ptrs[] = {x, weight, bias, conv_state_in, conv_state_out, y, cu_seqlens};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(!ptr || aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: every pointer must be 16-byte aligned", fn);
    const size_t xbytes = (size_t)rows * D * (x_dtype == KDA_BF16 ? 2 : 4);
    const size_t ybytes = (size_t)rows * D * (y_dtype == KDA_BF16 ? 2 : 4);
    KDA_REQUIRE(rows == 0 || (const char *)y + ybytes <= (const char *)x || (const char *)x + xbytes <= (const char *)y,
                KDA_ERR_INVALID_ARG, "%s: y must not overlap x", fn);
    int N = B;
    if (cu_seqlens) {
        KDA_REQUIRE(B == 1 && n_seqs > 0, KDA_ERR_INVALID_ARG, "%s: varlen needs B == 1 and n_seqs > 0", fn);
        if (cu_seqlens_host) {
            KDA_REQUIRE(cu_seqlens_host[0] == 0, KDA_ERR_INVALID_ARG, "%s: cu_seqlens[0] must be 0", fn);
            for (int i = 0; i < n_seqs; ++i)
                KDA_REQUIRE(cu_seqlens_host[i + 1] >= cu_seqlens_host[i], KDA_ERR_INVALID_ARG,
                            "%s: cu_seqlens must not decrease (entry %d)", fn, i + 1);
            KDA_REQUIRE(cu_seqlens_host[n_seqs] == T, KDA_ERR_INVALID_ARG, "%s: cu_seqlens[n_seqs] = %d but T = %d",
                        fn, cu_seqlens_host[n_seqs], T);
        }
        N = n_seqs;
    } else {
        KDA_REQUIRE(!cu_seqlens_host, KDA_ERR_INVALID_ARG, "%s: cu_seqlens_host given without cu_seqlens", fn);
    }
    if (conv_state_in && conv_state_out) {
        const size_t sbytes = (size_t)N * (W - 1) * D * sizeof(float);
        const char *a = (const char *)conv_state_in, *b = (const char *)conv_state_out;
        const bool overlap = a < b + sbytes && b < a + sbytes;
        KDA_REQUIRE(!overlap || (a == b && !cu_seqlens && T == 1), KDA_ERR_INVALID_ARG,
                    "%s: conv_state_out may alias conv_state_in only for a decode step (dense, T = 1)", fn);
    }
    return kda::launch_short_conv(x, x_dtype == KDA_BF16, weight, bias, conv_state_in, conv_state_out, y,
                                  y_dtype == KDA_BF16, cu_seqlens, N, rows, T, D, W, activation,
                                  (cudaStream_t)stream);
}

kda_status kda_o_proj(const void *y, const void *w_o, void *out, kda_dtype out_dtype, int64_t rows,
                      int in_features, int out_features, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_o_proj";
    KDA_REQUIRE(rows >= 0 && in_features > 0 && out_features > 0, KDA_ERR_INVALID_ARG,
                "%s: need rows >= 0 and positive feature counts", fn);
    KDA_REQUIRE(rows == 0 || (y && w_o && out), KDA_ERR_INVALID_ARG, "%s: y, w_o and out must not be NULL", fn);
    KDA_REQUIRE(dtype_ok(out_dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported out dtype", fn);
    KDA_REQUIRE(kda::o_proj_supported(in_features, out_features), KDA_ERR_UNSUPPORTED,
                "%s: in_features must be a multiple of 64 and out_features a multiple of 128", fn);
    KDA_REQUIRE(rows <= INT32_MAX, KDA_ERR_INVALID_ARG, "%s: too many rows", fn);
    const void *ptrs[] = {y, w_o, out};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(!ptr || aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: every pointer must be 16-byte aligned", fn);
    if (rows == 0) return KDA_OK;
    {
        const size_t r = (size_t)rows, ob = out_dtype == KDA_BF16 ? 2 : 4;
        const Span o{out, r * out_features * ob, "out"};
        KDA_REQUIRE(!overlaps(o, Span{y, r * in_features * 2, "y"}) &&
                        !overlaps(o, Span{w_o, (size_t)out_features * in_features * 2, "w_o"}),
                    KDA_ERR_INVALID_ARG, "%s: out must not overlap y or w_o", fn);
    }
    return kda::launch_o_proj(y, w_o, out, out_dtype == KDA_BF16, rows, in_features, out_features,
                              (cudaStream_t)stream);
}

kda_status kda_rotary(const void *x, kda_dtype dtype, int64_t x_stride, const int32_t *positions,
                      const double *inv_freq, float magnitude, int rotary_dim, int layout, int inverse, void *out,
                      int64_t out_stride, int64_t tokens, int heads, int dim, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_rotary";
    KDA_REQUIRE(tokens >= 0 && heads > 0 && dim > 0, KDA_ERR_INVALID_ARG, "%s: need tokens >= 0, heads > 0, dim > 0",
                fn);
    KDA_REQUIRE(dtype_ok(dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported dtype", fn);
    KDA_REQUIRE(dim % 8 == 0 && dim <= 256, KDA_ERR_UNSUPPORTED, "%s: dim=%d must be a multiple of 8, at most 256", fn,
                dim);
    KDA_REQUIRE(heads <= (1 << 20) && tokens <= INT32_MAX, KDA_ERR_UNSUPPORTED, "%s: too many heads or tokens", fn);
    KDA_REQUIRE(rotary_dim > 0, KDA_ERR_INVALID_ARG, "%s: rotary_dim must be positive", fn);
    kda_status s = check_rotary_args(fn, inv_freq, magnitude, rotary_dim, layout, dim);
    if (s != KDA_OK) return s;
    KDA_REQUIRE(inverse == 0 || inverse == 1, KDA_ERR_INVALID_ARG, "%s: inverse must be 0 or 1", fn);
    KDA_REQUIRE(tokens == 0 || (x && out && positions), KDA_ERR_INVALID_ARG,
                "%s: x, positions and out must not be NULL", fn);
    const int64_t row = (int64_t)heads * dim;
    if ((s = check_stride(fn, "x", x_stride, row, esize(dtype))) != KDA_OK) return s;
    if ((s = check_stride(fn, "out", out_stride, row, esize(dtype))) != KDA_OK) return s;
    KDA_REQUIRE(aligned16(x) && aligned16(out) && aligned_to(positions, 4), KDA_ERR_INVALID_ARG,
                "%s: x and out must be 16-byte aligned, positions 4-byte", fn);
    const Span in[] = {{positions, (size_t)tokens * 4, "positions"},
                       {inv_freq, (size_t)rotary_dim / 2 * 8, "inv_freq"},
                       {x == out && x_stride == out_stride ? nullptr : x,
                        strided_bytes(tokens, row, x_stride, esize(dtype)), "x"}};
    const Span o[] = {{out, strided_bytes(tokens, row, out_stride, esize(dtype)), "out"}};
    if ((s = check_apart(fn, in, 3, o, 1)) != KDA_OK) return s;
    kda::RotaryParams r;
    r.inv_freq = inv_freq;
    r.magnitude = magnitude;
    r.R = rotary_dim;
    r.interleaved = layout == KDA_ROTARY_INTERLEAVED;
    r.sign = inverse ? -1.f : 1.f;
    return kda::launch_rotary(x, dtype == KDA_BF16, x_stride, positions, r, out, out_stride, tokens, heads, dim,
                              (cudaStream_t)stream);
}

kda_status kda_kv_append(const void *k, int64_t k_stride, const void *v, int64_t v_stride, int64_t tokens,
                         int kv_heads, int dim, void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                         int num_pages, int page_size, const int32_t *block_table, int max_blocks,
                         const int32_t *context_lens, const int32_t *cu_seqlens, int n_seqs, const double *inv_freq,
                         float magnitude, int rotary_dim, int layout, const void *q, int64_t q_stride, int q_heads,
                         void *q_out, void *k_out, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_kv_append";
    kda_status s = check_cache_args(fn, k_cache, v_cache, k_scale, v_scale, num_pages, page_size, block_table,
                                    max_blocks, context_lens, n_seqs, q ? q_heads : kv_heads, kv_heads, dim);
    if (s != KDA_OK) return s;
    if ((s = check_rotary_args(fn, inv_freq, magnitude, rotary_dim, layout, dim)) != KDA_OK) return s;
    KDA_REQUIRE(tokens >= 0 && tokens <= INT32_MAX, KDA_ERR_INVALID_ARG, "%s: need 0 <= tokens < 2^31", fn);
    KDA_REQUIRE(tokens == 0 || (k && v), KDA_ERR_INVALID_ARG, "%s: k and v must not be NULL", fn);
    KDA_REQUIRE((q != nullptr) == (q_out != nullptr), KDA_ERR_INVALID_ARG, "%s: q and q_out come together", fn);
    KDA_REQUIRE(!q || q_heads > 0, KDA_ERR_INVALID_ARG, "%s: q needs q_heads > 0", fn);
    KDA_REQUIRE(tokens == 0 || n_seqs > 0, KDA_ERR_INVALID_ARG, "%s: tokens without sequences", fn);
    KDA_REQUIRE(cu_seqlens || tokens == n_seqs, KDA_ERR_INVALID_ARG,
                "%s: without cu_seqlens there is one token per sequence (tokens=%lld, n_seqs=%d)", fn, (long long)tokens,
                n_seqs);
    const int64_t kr = (int64_t)kv_heads * dim, qr = (int64_t)q_heads * dim;
    if ((s = check_stride(fn, "k", k_stride, kr, 2)) != KDA_OK) return s;
    if ((s = check_stride(fn, "v", v_stride, kr, 2)) != KDA_OK) return s;
    if (q && (s = check_stride(fn, "q", q_stride, qr, 2)) != KDA_OK) return s;
    const void *ptrs[] = {k, v, q, q_out, k_out};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: k, v, q, q_out and k_out must be 16-byte aligned", fn);
    KDA_REQUIRE(aligned_to(cu_seqlens, 4), KDA_ERR_INVALID_ARG, "%s: cu_seqlens must be 4-byte aligned", fn);
    const size_t blocks = (size_t)num_pages * kv_heads, codes = blocks * page_size * dim;
    const Span in[] = {{k, strided_bytes(tokens, kr, k_stride, 2), "k"},
                       {v, strided_bytes(tokens, kr, v_stride, 2), "v"},
                       {q, q ? strided_bytes(tokens, qr, q_stride, 2) : 0, "q"},
                       {block_table, (size_t)n_seqs * max_blocks * 4, "block_table"},
                       {context_lens, (size_t)n_seqs * 4, "context_lens"},
                       {cu_seqlens, ((size_t)n_seqs + 1) * 4, "cu_seqlens"},
                       {inv_freq, (size_t)rotary_dim / 2 * 8, "inv_freq"}};
    const Span out[] = {{k_cache, codes, "k_cache"},
                        {v_cache, codes, "v_cache"},
                        {k_scale, blocks * 4, "k_scale"},
                        {v_scale, blocks * 4, "v_scale"},
                        {q_out, q_out ? (size_t)tokens * qr * 2 : 0, "q_out"},
                        {k_out, (size_t)tokens * kr * 2, "k_out"}};
    if ((s = check_apart(fn, in, 7, out, 6)) != KDA_OK) return s;
    kda::AppendParams p;
    p.c = kda::PagedCache{static_cast<uint8_t *>(k_cache), static_cast<uint8_t *>(v_cache), k_scale, v_scale,
                          block_table, context_lens, num_pages, max_blocks, kv_heads, page_size, dim, n_seqs, __builtin_ctz(page_size)};
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu_seqlens = cu_seqlens;
    p.tokens = tokens;
    p.rot = kda::RotaryParams{inv_freq, magnitude, rotary_dim, layout == KDA_ROTARY_INTERLEAVED, 1.f};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.Hq = q ? q_heads : 0;
    p.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.k_out = static_cast<__nv_bfloat16 *>(k_out);
    return kda::launch_kv_append(p, (cudaStream_t)stream);
}

size_t kda_attn_decode_workspace_size(int n_seqs, int q_heads, int kv_heads, int dim, int64_t max_tokens) {
    if (n_seqs < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || (dim != 64 && dim != 128) ||
        max_tokens < 0 || max_tokens > INT32_MAX)
        return 0;
    return kda::attn_decode_workspace_bytes(n_seqs, q_heads, kv_heads, dim, max_tokens);
}

kda_status kda_attn_decode(const void *q, int64_t q_stride, const void *k_cache, const void *v_cache,
                           const float *k_scale, const float *v_scale, int num_pages, int page_size,
                           const int32_t *block_table, int max_blocks, const int32_t *seq_lens, int n_seqs,
                           int q_heads, int kv_heads, int dim, float scale, void *o, kda_dtype o_dtype, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_attn_decode";
    KDA_REQUIRE(q_heads > 0, KDA_ERR_INVALID_ARG, "%s: need q_heads > 0", fn);
    kda_status s = check_cache_args(fn, k_cache, v_cache, k_scale, v_scale, num_pages, page_size, block_table,
                                    max_blocks, seq_lens, n_seqs, q_heads, kv_heads, dim);
    if (s != KDA_OK) return s;
    KDA_REQUIRE(dtype_ok(o_dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported dtype", fn);
    KDA_REQUIRE(std::isfinite(scale), KDA_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    KDA_REQUIRE(n_seqs == 0 || (q && o), KDA_ERR_INVALID_ARG, "%s: q and o must not be NULL", fn);
    const int64_t row = (int64_t)q_heads * dim;
    if ((s = check_stride(fn, "q", q_stride, row, 2)) != KDA_OK) return s;
    const void *ptrs[] = {q, o, workspace};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: q, o and the workspace must be 16-byte aligned", fn);
    KDA_REQUIRE(aligned_to(lse, 4), KDA_ERR_INVALID_ARG, "%s: lse must be 4-byte aligned", fn);
    if (n_seqs == 0) return KDA_OK;
    const size_t need =
        kda::attn_decode_workspace_bytes(n_seqs, q_heads, kv_heads, dim, (int64_t)max_blocks * page_size);
    KDA_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), KDA_ERR_INVALID_ARG,
                "%s: the workspace holds %zu bytes, this call needs %zu (kda_attn_decode_workspace_size)", fn,
                workspace ? workspace_bytes : (size_t)0, need);
    const size_t blocks = (size_t)num_pages * kv_heads, codes = blocks * page_size * dim;
    const Span in[] = {{q, strided_bytes(n_seqs, row, q_stride, 2), "q"},
                       {k_cache, codes, "k_cache"},
                       {v_cache, codes, "v_cache"},
                       {k_scale, blocks * 4, "k_scale"},
                       {v_scale, blocks * 4, "v_scale"},
                       {block_table, (size_t)n_seqs * max_blocks * 4, "block_table"},
                       {seq_lens, (size_t)n_seqs * 4, "seq_lens"}};
    const Span out[] = {{o, (size_t)n_seqs * row * esize(o_dtype), "o"},
                        {lse, (size_t)n_seqs * q_heads * 4, "lse"},
                        {workspace, need, "the workspace"}};
    if ((s = check_apart(fn, in, 7, out, 3)) != KDA_OK) return s;
    kda::DecodeParams p;
    p.c = kda::PagedCache{static_cast<uint8_t *>(const_cast<void *>(k_cache)),
                          static_cast<uint8_t *>(const_cast<void *>(v_cache)), const_cast<float *>(k_scale),
                          const_cast<float *>(v_scale), block_table, seq_lens, num_pages, max_blocks, kv_heads,
                          page_size, dim, n_seqs, __builtin_ctz(page_size)};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.Hq = q_heads;
    p.scale = scale;
    p.o = o;
    p.o_bf16 = o_dtype == KDA_BF16;
    p.lse = lse;
    p.ws = static_cast<float *>(workspace);
    p.whole = 0;
    p.polls = std::min(kda::wait_polls(), kda::kAttnPolls);
    return kda::launch_attn_decode(p, (cudaStream_t)stream);
}

size_t kda_attn_prompt_workspace_size(int64_t q_rows, int64_t k_rows, int q_heads, int kv_heads, int dim_v, int n_seqs) {
    if (q_rows <= 0 || q_rows > (1 << 30) || k_rows < 0 || k_rows > (1 << 30) || q_heads <= 0 || q_heads > 65535 ||
        kv_heads <= 0 || q_heads % kv_heads != 0 || n_seqs <= 0 || n_seqs > 16384 || (dim_v != 64 && dim_v != 128))
        return 0;
    return kda::attn_prompt_workspace_bytes(q_rows, k_rows, n_seqs, q_heads, kv_heads, dim_v);
}

kda_status kda_attn_prompt(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, int64_t q_rows, int64_t k_rows, int q_heads, int kv_heads, int dim,
                           int dim_v, const int32_t *cu_seqlens, const int32_t *cu_seqlens_k, int n_seqs, float scale,
                           void *o, kda_dtype o_dtype, float *lse, void *workspace, size_t workspace_bytes,
                           void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_attn_prompt";
    KDA_REQUIRE(q_rows >= 0 && k_rows >= 0 && q_heads > 0 && kv_heads > 0 && n_seqs >= 0, KDA_ERR_INVALID_ARG,
                "%s: need rows >= 0, heads > 0, n_seqs >= 0", fn);
    KDA_REQUIRE((dim == 64 && dim_v == 64) || (dim == 128 && dim_v == 128) || (dim == 192 && dim_v == 128),
                KDA_ERR_UNSUPPORTED, "%s: dim=%d dim_v=%d (supported: 64/64, 128/128, 192/128)", fn, dim, dim_v);
    KDA_REQUIRE(q_heads % kv_heads == 0, KDA_ERR_INVALID_ARG, "%s: q_heads=%d is not a multiple of kv_heads=%d", fn,
                q_heads, kv_heads);
    KDA_REQUIRE(q_rows <= (1 << 30) && k_rows <= (1 << 30) && q_heads <= 65535, KDA_ERR_UNSUPPORTED,
                "%s: at most 2^30 rows and 65535 heads", fn);
    KDA_REQUIRE(n_seqs <= 16384, KDA_ERR_UNSUPPORTED, "%s: at most 16384 sequences", fn);
    KDA_REQUIRE(dtype_ok(o_dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported dtype", fn);
    KDA_REQUIRE(std::isfinite(scale) && scale != 0.f, KDA_ERR_INVALID_ARG, "%s: scale must be finite and not 0", fn);
    KDA_REQUIRE(q_rows == 0 || (q && o), KDA_ERR_INVALID_ARG, "%s: q and o must not be NULL", fn);
    KDA_REQUIRE(k_rows == 0 || (k && v), KDA_ERR_INVALID_ARG, "%s: k and v must not be NULL", fn);
    KDA_REQUIRE(q_rows == 0 || n_seqs > 0, KDA_ERR_INVALID_ARG, "%s: rows without sequences", fn);
    if (!cu_seqlens) {
        KDA_REQUIRE(!cu_seqlens_k, KDA_ERR_INVALID_ARG, "%s: cu_seqlens_k without cu_seqlens", fn);
        KDA_REQUIRE(n_seqs == 0 || (q_rows % n_seqs == 0 && k_rows % n_seqs == 0), KDA_ERR_INVALID_ARG,
                    "%s: without cu_seqlens the rows must divide into n_seqs equal sequences", fn);
    } else {
        KDA_REQUIRE(cu_seqlens_k || q_rows == k_rows, KDA_ERR_INVALID_ARG,
                    "%s: without cu_seqlens_k there are as many keys as queries", fn);
    }
    const int64_t qr = (int64_t)q_heads * dim, kr = (int64_t)kv_heads * dim, vr = (int64_t)kv_heads * dim_v,
                  orow = (int64_t)q_heads * dim_v;
    kda_status s;
    if ((s = check_stride(fn, "q", q_stride, qr, 2)) != KDA_OK) return s;
    if ((s = check_stride(fn, "k", k_stride, kr, 2)) != KDA_OK) return s;
    if ((s = check_stride(fn, "v", v_stride, vr, 2)) != KDA_OK) return s;
    const void *ptrs[] = {q, k, v, o};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: q, k, v and o must be 16-byte aligned", fn);
    KDA_REQUIRE(aligned_to(lse, 4) && aligned_to(cu_seqlens, 4) && aligned_to(cu_seqlens_k, 4), KDA_ERR_INVALID_ARG,
                "%s: lse and cu_seqlens must be 4-byte aligned", fn);
    KDA_REQUIRE(aligned16(workspace), KDA_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned", fn);
    if (q_rows == 0) return KDA_OK;
    const size_t need = kda::attn_prompt_workspace_bytes(q_rows, k_rows, n_seqs, q_heads, kv_heads, dim_v);
    KDA_REQUIRE(!workspace || workspace_bytes >= need, KDA_ERR_INVALID_ARG,
                "%s: the workspace holds %zu bytes, this call uses %zu (kda_attn_prompt_workspace_size)", fn,
                workspace_bytes, need);
    const size_t cu_bytes = ((size_t)n_seqs + 1) * 4;
    const Span in[] = {{q, strided_bytes(q_rows, qr, q_stride, 2), "q"},
                       {k, strided_bytes(k_rows, kr, k_stride, 2), "k"},
                       {v, strided_bytes(k_rows, vr, v_stride, 2), "v"},
                       {cu_seqlens, cu_bytes, "cu_seqlens"},
                       {cu_seqlens_k, cu_bytes, "cu_seqlens_k"}};
    const Span out[] = {{o, (size_t)q_rows * orow * esize(o_dtype), "o"}, {lse, (size_t)q_rows * q_heads * 4, "lse"},
                        {workspace, need, "the workspace"}};
    if ((s = check_apart(fn, in, 5, out, 3)) != KDA_OK) return s;
    kda::PromptParams p;
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu_q = cu_seqlens;
    p.cu_k = cu_seqlens_k ? cu_seqlens_k : cu_seqlens;
    p.Tq = q_rows;
    p.Tk = k_rows;
    p.N = n_seqs;
    p.Hq = q_heads;
    p.Hk = kv_heads;
    p.D = dim;
    p.DV = dim_v;
    p.scale = scale;
    p.o = o;
    p.o_bf16 = o_dtype == KDA_BF16;
    p.lse = lse;
    p.ws = need ? static_cast<float *>(workspace) : nullptr;
    p.polls = std::min(kda::wait_polls(), kda::kAttnPolls);
    return kda::launch_attn_prompt(p, (cudaStream_t)stream);
}

kda_status kda_latent_append(const void *x, int64_t x_stride, int64_t tokens, void *cache, int num_pages, int page_size,
                             const int32_t *block_table, int max_blocks, const int32_t *context_lens,
                             const int32_t *cu_seqlens, int n_seqs, const float *norm_w, float eps, const double *inv_freq,
                             float magnitude, int rotary_dim, int layout, void *rows_out, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_latent_append";
    kda_status s = check_latent_cache(fn, cache, num_pages, page_size, block_table, max_blocks, context_lens, cu_seqlens, n_seqs,
                                      tokens);
    if (s != KDA_OK) return s;
    if ((s = check_rotary_args(fn, inv_freq, magnitude, rotary_dim, layout, kda::kShared)) != KDA_OK) return s;
    KDA_REQUIRE(tokens == 0 || x, KDA_ERR_INVALID_ARG, "%s: x must not be NULL", fn);
    // (2^-100: mean(c^2) + eps keeps its precision down to the smallest sums that fp32 holds)
    KDA_REQUIRE(!norm_w || (std::isfinite(eps) && eps >= 7.888609052210118e-31f), KDA_ERR_INVALID_ARG,
                "%s: eps must be finite and at least 2^-100", fn);
    KDA_REQUIRE(aligned16(x) && aligned16(rows_out), KDA_ERR_INVALID_ARG, "%s: x and rows_out must be 16-byte aligned", fn);
    KDA_REQUIRE(aligned_to(norm_w, 4), KDA_ERR_INVALID_ARG, "%s: norm_w must be 4-byte aligned", fn);
    if ((s = check_stride(fn, "x", x_stride, kda::kRow, 2)) != KDA_OK) return s;
    const Span in[] = {{x, strided_bytes(tokens, kda::kRow, x_stride, 2), "x"},
                       {block_table, (size_t)n_seqs * max_blocks * 4, "block_table"},
                       {context_lens, (size_t)n_seqs * 4, "context_lens"},
                       {cu_seqlens, ((size_t)n_seqs + 1) * 4, "cu_seqlens"},
                       {norm_w, (size_t)kda::kLatent * 4, "norm_w"},
                       {inv_freq, (size_t)rotary_dim / 2 * 8, "inv_freq"}};
    const Span out[] = {{cache, (size_t)num_pages * page_size * kda::kRow * 2, "the cache"},
                        {rows_out, (size_t)tokens * kda::kRow * 2, "rows_out"}};
    if ((s = check_apart(fn, in, 6, out, 2)) != KDA_OK) return s;
    kda::LatentAppendParams p;
    p.c = kda::LatentCache{static_cast<__nv_bfloat16 *>(cache), block_table, context_lens, num_pages, max_blocks, page_size,
                           n_seqs, __builtin_ctz(page_size)};
    p.x = static_cast<const __nv_bfloat16 *>(x);
    p.x_stride = x_stride;
    p.tokens = tokens;
    p.cu_seqlens = cu_seqlens;
    p.norm_w = norm_w;
    p.eps = eps;
    p.rot = kda::RotaryParams{inv_freq, magnitude, rotary_dim, layout == KDA_ROTARY_INTERLEAVED, 1.f};
    p.rows_out = static_cast<__nv_bfloat16 *>(rows_out);
    return kda::launch_latent_append(p, (cudaStream_t)stream);
}

kda_status kda_latent_queries(const void *q, int64_t q_stride, int64_t tokens, int heads, const void *w_kv,
                              const int32_t *positions, const double *inv_freq, float magnitude, int rotary_dim, int layout,
                              void *out, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_latent_queries";
    const int64_t row = (int64_t)heads * kda::kHeadQuery;
    kda_status s = check_latent_product(fn, q, "q", q_stride, row, tokens, heads, w_kv, out, out);
    if (s != KDA_OK) return s;
    if ((s = check_rotary_args(fn, inv_freq, magnitude, rotary_dim, layout, kda::kShared)) != KDA_OK) return s;
    KDA_REQUIRE(tokens == 0 || (rotary_dim > 0) == (positions != nullptr), KDA_ERR_INVALID_ARG,
                "%s: positions and inv_freq come together", fn);
    KDA_REQUIRE(aligned_to(positions, 4), KDA_ERR_INVALID_ARG, "%s: positions must be 4-byte aligned", fn);
    const Span in[] = {{q, strided_bytes(tokens, row, q_stride, 2), "q"},
                       {w_kv, (size_t)heads * 256 * kda::kLatent * 2, "w_kv"},
                       {positions, (size_t)tokens * 4, "positions"},
                       {inv_freq, (size_t)rotary_dim / 2 * 8, "inv_freq"}};
    const Span outs[] = {{out, (size_t)tokens * heads * kda::kRow * 2, "out"}};
    if ((s = check_apart(fn, in, 4, outs, 1)) != KDA_OK) return s;
    kda::LatentProductParams p = {};
    p.what = kda::kLatentQueries;
    p.x = static_cast<const __nv_bfloat16 *>(q);
    p.x_stride = q_stride;
    p.tokens = tokens;
    p.H = heads;
    p.w = static_cast<const __nv_bfloat16 *>(w_kv);
    p.positions = positions;
    p.rot = kda::RotaryParams{inv_freq, magnitude, rotary_dim, layout == KDA_ROTARY_INTERLEAVED, 1.f};
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.polls = std::min(kda::wait_polls(), kda::kAttnPolls);
    return kda::launch_latent_product(p, (cudaStream_t)stream);
}

kda_status kda_latent_values(const void *o, int64_t o_stride, int64_t tokens, int heads, const void *w_kv, void *out,
                             void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_latent_values";
    const int64_t row = (int64_t)heads * kda::kLatent;
    kda_status s = check_latent_product(fn, o, "o", o_stride, row, tokens, heads, w_kv, out, out);
    if (s != KDA_OK) return s;
    const Span in[] = {{o, strided_bytes(tokens, row, o_stride, 2), "o"}, {w_kv, (size_t)heads * 256 * kda::kLatent * 2, "w_kv"}};
    const Span outs[] = {{out, (size_t)tokens * heads * kda::kHeadValue * 2, "out"}};
    if ((s = check_apart(fn, in, 2, outs, 1)) != KDA_OK) return s;
    kda::LatentProductParams p = {};
    p.what = kda::kLatentValues;
    p.x = static_cast<const __nv_bfloat16 *>(o);
    p.x_stride = o_stride;
    p.tokens = tokens;
    p.H = heads;
    p.w = static_cast<const __nv_bfloat16 *>(w_kv);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.polls = std::min(kda::wait_polls(), kda::kAttnPolls);
    return kda::launch_latent_product(p, (cudaStream_t)stream);
}

kda_status kda_latent_expand(const void *rows, int64_t rows_stride, int64_t tokens, int heads, const void *w_kv, void *k,
                             void *v, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_latent_expand";
    kda_status s = check_latent_product(fn, rows, "rows", rows_stride, kda::kRow, tokens, heads, w_kv, k, v);
    if (s != KDA_OK) return s;
    const Span in[] = {{rows, strided_bytes(tokens, kda::kRow, rows_stride, 2), "rows"},
                       {w_kv, (size_t)heads * 256 * kda::kLatent * 2, "w_kv"}};
    const Span outs[] = {{k, (size_t)tokens * heads * kda::kHeadQuery * 2, "k"}, {v, (size_t)tokens * heads * kda::kHeadValue * 2, "v"}};
    if ((s = check_apart(fn, in, 2, outs, 2)) != KDA_OK) return s;
    kda::LatentProductParams p = {};
    p.what = kda::kLatentExpand;
    p.x = static_cast<const __nv_bfloat16 *>(rows);
    p.x_stride = rows_stride;
    p.tokens = tokens;
    p.H = heads;
    p.w = static_cast<const __nv_bfloat16 *>(w_kv);
    p.out = static_cast<__nv_bfloat16 *>(k);
    p.out2 = static_cast<__nv_bfloat16 *>(v);
    p.polls = std::min(kda::wait_polls(), kda::kAttnPolls);
    return kda::launch_latent_product(p, (cudaStream_t)stream);
}

size_t kda_attn_latent_workspace_size(int n_seqs, int64_t tokens, int heads, int64_t max_tokens) {
    if (n_seqs <= 0 || n_seqs > 65535 || tokens <= 0 || tokens > (1 << 24) || heads <= 0 || heads > 4096 || max_tokens < 0 ||
        max_tokens > INT32_MAX - 256)
        return 0;
    return kda::attn_latent_workspace_bytes(n_seqs, tokens, heads, max_tokens);
}

kda_status kda_attn_latent(const void *q, int64_t q_stride, int64_t tokens, int heads, const void *cache, int num_pages,
                           int page_size, const int32_t *block_table, int max_blocks, const int32_t *seq_lens,
                           const int32_t *cu_seqlens, int n_seqs, float scale, void *o, kda_dtype o_dtype, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream) {
    kda::g_err[0] = 0;
    const char *fn = "kda_attn_latent";
    kda_status s = check_latent_cache(fn, cache, num_pages, page_size, block_table, max_blocks, seq_lens, cu_seqlens, n_seqs,
                                      tokens);
    if (s != KDA_OK) return s;
    KDA_REQUIRE(heads > 0, KDA_ERR_INVALID_ARG, "%s: need heads > 0", fn);
    KDA_REQUIRE(heads <= 4096 && tokens <= (1 << 24), KDA_ERR_UNSUPPORTED, "%s: at most 4096 heads and 2^24 tokens", fn);
    KDA_REQUIRE(dtype_ok(o_dtype), KDA_ERR_UNSUPPORTED, "%s: unsupported dtype", fn);
    KDA_REQUIRE(scale != 0.f && std::fabs(scale) <= 1.2676506002282294e30f, KDA_ERR_INVALID_ARG,
                "%s: scale must not be 0 and lie within 2^100", fn);
    KDA_REQUIRE(tokens == 0 || (q && o), KDA_ERR_INVALID_ARG, "%s: q and o must not be NULL", fn);
    const int64_t row = (int64_t)heads * kda::kRow;
    if ((s = check_stride(fn, "q", q_stride, row, 2)) != KDA_OK) return s;
    const void *ptrs[] = {q, o, workspace};
    for (const void *ptr : ptrs)
        KDA_REQUIRE(aligned16(ptr), KDA_ERR_INVALID_ARG, "%s: q, o and the workspace must be 16-byte aligned", fn);
    KDA_REQUIRE(aligned_to(lse, 4), KDA_ERR_INVALID_ARG, "%s: lse must be 4-byte aligned", fn);
    if (tokens == 0) return KDA_OK;
    const size_t need = kda::attn_latent_workspace_bytes(n_seqs, tokens, heads, (int64_t)max_blocks * page_size);
    KDA_REQUIRE(need == 0 || (workspace && workspace_bytes >= need), KDA_ERR_INVALID_ARG,
                "%s: the workspace holds %zu bytes, this call needs %zu (kda_attn_latent_workspace_size)", fn,
                workspace ? workspace_bytes : (size_t)0, need);
    const Span in[] = {{q, strided_bytes(tokens, row, q_stride, 2), "q"},
                       {cache, (size_t)num_pages * page_size * kda::kRow * 2, "the cache"},
                       {block_table, (size_t)n_seqs * max_blocks * 4, "block_table"},
                       {seq_lens, (size_t)n_seqs * 4, "seq_lens"},
                       {cu_seqlens, ((size_t)n_seqs + 1) * 4, "cu_seqlens"}};
    const Span out[] = {{o, (size_t)tokens * heads * kda::kLatent * esize(o_dtype), "o"},
                        {lse, (size_t)tokens * heads * 4, "lse"},
                        {workspace, need, "the workspace"}};
    if ((s = check_apart(fn, in, 5, out, 3)) != KDA_OK) return s;
    kda::AttnLatentParams p;
    p.c = kda::LatentCache{static_cast<__nv_bfloat16 *>(const_cast<void *>(cache)), block_table, seq_lens, num_pages, max_blocks,
                           page_size, n_seqs, __builtin_ctz(page_size)};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.q_stride = q_stride;
    p.tokens = (int)tokens;
    p.H = heads;
    p.cu_seqlens = cu_seqlens;
    p.scale = scale;
    p.o = o;
    p.o_bf16 = o_dtype == KDA_BF16;
    p.lse = lse;
    p.ws = static_cast<float *>(workspace);
    p.polls = std::min(kda::wait_polls(), kda::kAttnPolls);
    return kda::launch_attn_latent(p, (cudaStream_t)stream);
}

}  // extern "C"
