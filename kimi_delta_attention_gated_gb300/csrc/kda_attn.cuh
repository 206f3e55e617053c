// kda_attn.cuh -- definitions shared by the full-attention operators: the position
// rotation (kda_rotary.cu), the paged 8-bit key/value cache and its append
// (kda_kv_append.cu), single-token attention over it (kda_attn_decode.cu) and the prompt's
// attention (kda_attn_prompt.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "kda_internal.cuh"

namespace kda {

// ---------------------------------------------------------------------------
// parameter blocks

struct RotaryParams {
    const double *inv_freq;  // [R / 2] radians per position, or null: no rotation
    float magnitude;         // factor on the rotated channels
    int R;                   // rotated channels: the first R of a head
    int interleaved;         // pairs (2i, 2i + 1); else (i, i + R / 2)
    float sign;              // -1: the transposed rotation
};

struct PagedCache {
    uint8_t *k, *v;               // e4m3 codes [pages, Hk, P, D]
    float *k_scale, *v_scale;     // [pages, Hk]
    const int32_t *block_table;   // [N, max_blocks]
    const int32_t *lens;          // [N] tokens in the cache
    int n_pages, max_blocks, Hk, P, D, N;
    int p_shift;                  // P = 1 << p_shift
};

struct AppendParams {
    PagedCache c;                 // lens: tokens before this call
    const __nv_bfloat16 *k, *v;   // rows of Hk * D, k_stride / v_stride elements apart
    int64_t k_stride, v_stride;
    const int32_t *cu_seqlens;    // [N + 1] or null: one token per sequence
    int64_t tokens;
    RotaryParams rot;
    const __nv_bfloat16 *q;       // rows of Hq * D, or null
    int64_t q_stride;
    int Hq;
    __nv_bfloat16 *q_out, *k_out; // dense [tokens, Hq, D] / [tokens, Hk, D]; k_out may be null
};

// Bound on the attention kernels' waits, 8 s (a poll that finds nothing takes 3.8 us, measured): a
// CTA waits for nothing but its own warps and copies, none of which does work of unbounded length
// while another waits.  The first-line waits on copies take a lower one from kda_set_wait_limit.
constexpr uint32_t kAttnPolls = 1u << 21;

struct DecodeParams {
    PagedCache c;                 // lens: tokens in the cache
    const __nv_bfloat16 *q;       // rows of Hq * D, q_stride elements apart
    int64_t q_stride;
    int Hq;
    float scale;
    void *o;                      // [N, Hq, D]
    int o_bf16;
    float *lse;                   // [N, Hq] or null
    float *ws;                    // partial results
    int whole;                    // a CTA for each (sequence, head), no partial results
    uint32_t polls;               // bound on the copies' waits
};

struct PromptParams {
    const __nv_bfloat16 *q, *k, *v;  // rows of Hq * D, Hk * D, Hk * DV
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_q, *cu_k;      // [N + 1], or null: N sequences of equal lengths
    int64_t Tq, Tk;
    int N, Hq, Hk, D, DV;
    float scale;
    void *o;                         // [Tq, Hq, DV]
    int o_bf16;
    float *lse;                      // [Tq, Hq] or null
    float *ws;                       // sums of parts of the keys, or null: every row's keys in one go
    uint32_t polls;                  // bound on the copies' waits
};

kda_status launch_rotary(const void *x, int bf16, int64_t x_stride, const int32_t *positions, const RotaryParams &r,
                         void *out, int64_t out_stride, int64_t T, int H, int D, cudaStream_t st);
kda_status launch_kv_append(const AppendParams &p, cudaStream_t st);
size_t attn_decode_workspace_bytes(int64_t N, int Hq, int Hk, int D, int64_t max_tokens);
kda_status launch_attn_decode(const DecodeParams &p, cudaStream_t st);
kda_status launch_attn_prompt(const PromptParams &p, cudaStream_t st);
size_t attn_prompt_workspace_bytes(int64_t Tq, int64_t Tk, int N, int Hq, int Hk, int DV);
int take_attn_prompt_timeouts(cudaStream_t st);
int take_attn_decode_timeouts(cudaStream_t st);

// ---------------------------------------------------------------------------
// angles

// One pair's turn per position as a 64-bit binary fraction of a full turn.  The fraction of
// position p is then the integer product p * turn modulo 2^64: the reduction to one turn is the
// integers' own wrap-around and loses nothing, so that the angle is off by the turn's own cut at
// 2^-64, p times (7e-10 rad at 2^31).  Formed from the double's 53-bit
// integer m and exponent with 64-bit integers (this GPU's double-precision rate is 1/50 of
// its integer rate): m * 2^e / (2 pi) = m * C * 2^(e - 66) with C = 2^66 / (2 pi).
__device__ __forceinline__ uint64_t turn_of(double inv_freq) {
    const uint64_t b = (uint64_t)__double_as_longlong(inv_freq);
    const int be = (int)(b >> 52) & 0x7FF;
    const uint64_t m = be == 0 ? 0ull : (b & 0xFFFFFFFFFFFFFull) | 1ull << 52;  // subnormals are no turn at all
    const uint64_t C = 11743562013128004906ull;
    const uint64_t hi = __umul64hi(m, C), lo = m * C;
    const int s = 2 - (be - 1075);  // the product's binary places behind the 64 that are kept
    const uint64_t t = s >= 128  ? 0ull
                       : s >= 64 ? hi >> (s - 64)
                       : s > 0   ? hi << (64 - s) | lo >> s
                       : s > -64 ? lo << -s
                                 : 0ull;
    return b >> 63 ? 0ull - t : t;
}

// cos and sin of 2 pi * f / 2^64.  f is split into the nearest quarter turn and a rest of at
// most 1/8 turn, taken as a + d, a the fp32 value of its first 32 bits and d what that and those
// bits leave out, so that the sine of a small angle has all its bits.  On |a| <= pi/4 the Taylor
// series through a^10 and a^9 leave 1e-9 of cos and sin; the last rounding is the only one that
// counts.
__device__ __forceinline__ void cos_sin_turn(uint64_t f, float &c, float &s) {
    const int low = (int)(uint32_t)f;  // signed: the first 32 bits are rounded
    const uint32_t top = (uint32_t)(f >> 32) + (low < 0);
    const uint32_t quarter = (top + (1u << 29)) >> 30;  // 4 is 0 again
    const int rest = (int)(top - (quarter << 30));
    constexpr float kHi = 1.4629180792671596e-9f;  // 2 pi / 2^32
    constexpr float kLo = (float)(6.283185307179586 / 4294967296.0 - (double)kHi);
    const float hi = (float)rest, lo = fmaf((float)low, 2.3283064365386963e-10f, (float)(rest - (int)hi));  // 2^-32
    const float a = hi * kHi;
    const float d = fmaf(hi, kHi, -a) + fmaf(hi, kLo, lo * kHi);
    const float a2 = a * a;
    float pc = -1.f / 3628800.f;
    pc = fmaf(pc, a2, 1.f / 40320.f);
    pc = fmaf(pc, a2, -1.f / 720.f);
    pc = fmaf(pc, a2, 1.f / 24.f);
    pc = fmaf(pc, a2, -0.5f);
    pc = 1.f + fmaf(pc, a2, -a * d);  // cos(a + d) = cos a - d sin a, sin a = a as far as it counts
    float ps = 1.f / 362880.f;
    ps = fmaf(ps, a2, -1.f / 5040.f);
    ps = fmaf(ps, a2, 1.f / 120.f);
    ps = fmaf(ps, a2, -1.f / 6.f);
    ps = a + fmaf(ps * a2, a, d);
    const float x = (quarter & 1) ? ps : pc, y = (quarter & 1) ? pc : ps;
    c = ((quarter + 1) & 2) ? -x : x;
    s = (quarter & 2) ? -y : y;
}

// a * b - c * d with the product's rounding error carried (two extra FMAs): within 1.5 ulp,
// so an 8-bit code chosen from it rarely differs from the exact value's.  An infinite product has
// no such error (inf - inf is NaN, of which fminf makes a number), and the difference stays infinite.
__device__ __forceinline__ float diff_of_products(float a, float b, float c, float d) {
    const float w = c * d;
    const float e = fmaf(-c, d, w);
    return fmaf(a, b, -w) + fminf(e, 3.4028234663852886e38f);
}

// The pair (a, b) turned: magnitude * (a cos - b sin, b cos + a sin).
__device__ __forceinline__ void turn_pair(float a, float b, float2 cs, float mag, float &x, float &y) {
    x = diff_of_products(a, cs.x, b, cs.y) * mag;
    y = diff_of_products(b, cs.x, -a, cs.y) * mag;
}

// ---------------------------------------------------------------------------
// 16-byte vectors of the two storage types as fp32

template <typename T>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ static void load(const uint4 &w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    __device__ static uint4 store(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Vec16<float> {
    static constexpr int N = 4;
    __device__ static void load(const uint4 &w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    __device__ static uint4 store(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// Where the cos / sin of pair j lie within a token's np pairs: eight consecutive pairs are
// read by one lane, two at a time, so pairs 8v + 2k, 8v + 2k + 1 of all v lie together.
__device__ __forceinline__ int cs_at(int j, int np) { return ((j >> 1) & 3) * (np >> 2) + (j >> 3) * 2 + (j & 1); }

// Pairs j and j + 1 (j even): 16 bytes.
__device__ __forceinline__ float4 cs_two(const float2 *cs, int j, int np) {
    return *reinterpret_cast<const float4 *>(cs + cs_at(j, np));
}

// cos / sin (times the sign) of `n` tokens' pairs into cs[token * np + cs_at(pair)]: a thread
// keeps to one pair, so its turn is formed once.
template <typename PosFn>
__device__ __forceinline__ void fill_cos_sin(float2 *cs, const RotaryParams &r, int n, PosFn pos, int tid, int threads) {
    const int np = r.R >> 1;
    if (np == 0) return;
    const int rows = threads / np, j = tid % np, row = tid / np;
    if (row >= rows) return;
    const uint64_t turn = turn_of(__ldg(r.inv_freq + j));
    cs += cs_at(j, np);
    for (int t = row; t < n; t += rows) {
        float c, s;
        cos_sin_turn((uint64_t)(int64_t)pos(t) * turn, c, s);
        cs[t * np] = make_float2(c, s * r.sign);
    }
}

// The same for n tokens at consecutive positions: the angle goes on by an integer addition.
__device__ __forceinline__ void fill_cos_sin_run(float2 *cs, const RotaryParams &r, int n, int64_t pos0, int tid,
                                                 int threads) {
    const int np = r.R >> 1, rows = threads / np, j = tid % np, row = tid / np;
    if (row >= rows) return;
    const uint64_t turn = turn_of(__ldg(r.inv_freq + j)), step = turn * (uint64_t)rows;
    uint64_t f = (uint64_t)(pos0 + row) * turn;
    cs += cs_at(j, np);
    for (int t = row; t < n; t += rows, f += step) {
        float c, s;
        cos_sin_turn(f, c, s);
        cs[t * np] = make_float2(c, s * r.sign);
    }
}

// Work units of one head: in the half layout a unit is two 16-byte vectors R / 2 channels
// apart, in the interleaved layout one vector; each vector behind the rotated part is one.
__host__ __device__ __forceinline__ int rotary_units(int D, int R, int interleaved, int vec) {
    return (interleaved ? R / vec : R / (2 * vec)) + (D - R) / vec;
}

// Unit u of one head: x -> y.
template <typename T>
__device__ __forceinline__ void rotate_unit(const T *x, T *y, const float2 *cs, int u, int R, int interleaved, float mag) {
    const int np = R >> 1;
    using V = Vec16<T>;
    constexpr int N = V::N;
    const int nrot = interleaved ? R / N : R / (2 * N);
    if (u >= nrot) {
        const int c = R + (u - nrot) * N;
        *reinterpret_cast<uint4 *>(y + c) = *reinterpret_cast<const uint4 *>(x + c);
        return;
    }
    float a[N];
    if (interleaved) {
        V::load(*reinterpret_cast<const uint4 *>(x + u * N), a);
        float o[N];
#pragma unroll
        for (int i = 0; i < N / 2; i += 2) {
            const float4 w = cs_two(cs, u * (N / 2) + i, np);
            turn_pair(a[2 * i], a[2 * i + 1], make_float2(w.x, w.y), mag, o[2 * i], o[2 * i + 1]);
            turn_pair(a[2 * i + 2], a[2 * i + 3], make_float2(w.z, w.w), mag, o[2 * i + 2], o[2 * i + 3]);
        }
        *reinterpret_cast<uint4 *>(y + u * N) = V::store(o);
    } else {
        float b[N], oa[N], ob[N];
        const uint4 wa = *reinterpret_cast<const uint4 *>(x + u * N);
        const uint4 wb = *reinterpret_cast<const uint4 *>(x + u * N + R / 2);
        V::load(wa, a);
        V::load(wb, b);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float4 w = cs_two(cs, u * N + i, np);
            turn_pair(a[i], b[i], make_float2(w.x, w.y), mag, oa[i], ob[i]);
            turn_pair(a[i + 1], b[i + 1], make_float2(w.z, w.w), mag, oa[i + 1], ob[i + 1]);
        }
        *reinterpret_cast<uint4 *>(y + u * N) = V::store(oa);
        *reinterpret_cast<uint4 *>(y + u * N + R / 2) = V::store(ob);
    }
}

// Rows of `n` tokens (token t at x + t * xs, y + t * ys, H heads of D) with cs filled.
template <typename T>
__device__ __forceinline__ void rotate_rows(const T *x, int64_t xs, T *y, int64_t ys, const float2 *cs,
                                            const RotaryParams &r, int n, int H, int D, int tid, int threads) {
    const int U = rotary_units(D, r.R, r.interleaved, Vec16<T>::N), per = H * U, np = r.R >> 1;
    // unit `tid` and then every threads-th, taken apart by additions
    const int dt = threads / per, dh = (threads - dt * per) / U, du = threads - dt * per - dh * U;
    int t = tid / per, h = (tid - t * per) / U, u = tid - t * per - h * U;
    while (t < n) {
        rotate_unit<T>(x + t * xs + h * D, y + t * ys + h * D, cs + t * np, u, r.R, r.interleaved, r.magnitude);
        t += dt;
        h += dh;
        u += du;
        if (u >= U) u -= U, ++h;
        if (h >= H) h -= H, ++t;
    }
}

// Tokens a CTA of `threads` rotates at once: about four 16-byte vectors a thread, at most
// what `room` cos / sin pairs of shared memory hold.
__host__ __device__ __forceinline__ int rotary_tile_tokens(int H, int D, int R, int vec, int threads, int room) {
    int n = threads * 4 * vec / (H * D);
    if (R > 0 && n > room / (R / 2)) n = room / (R / 2);
    return n < 1 ? 1 : n;
}

// ---------------------------------------------------------------------------
// e4m3

constexpr float kE4m3Max = 448.f;
constexpr int kScaleExpLo = -100, kScaleExpHi = 100;

// Two values as e4m3 codes, round to nearest even.  The block's scale keeps finite values
// within 448.  NaN stays NaN; an infinity has to become one (the type has none), which is
// looked at only where a block holds one.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float no_infinity(float x) { return isinf(x) ? __int_as_float(0x7fc00000) : x; }

__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// The smallest exponent e with amax <= 448 * 2^e, within the limits (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return amax > 0.f ? max(kScaleExpLo, min(kScaleExpHi, e)) : kScaleExpLo;
}

__device__ __forceinline__ int exp_of_scale(float s) {
    return max(kScaleExpLo, min(kScaleExpHi, (int)((__float_as_uint(s) >> 23) & 0xFFu) - 127));
}

// 4 codes multiplied by 2^d (d <= 0) and rounded to codes again.
__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float f) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        r |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x.x * f, x.y * f), __NV_SATFINITE, __NV_E4M3) << (16 * i);
    }
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float finite_abs(float x) {
    const float a = fabsf(x);
    return a <= 3.4028234663852886e38f ? a : 0.f;  // a NaN compares false
}

}  // namespace kda
