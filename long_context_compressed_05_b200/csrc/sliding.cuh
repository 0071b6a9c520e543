// Sliding-window layers: the key sets of prefill blocks and decode steps, the argument structs of the
// launchers, and the exponents and codes of 8-bit rows.
#pragma once

#include "internal.cuh"
#include "lowprec.cuh"

namespace hcsa {

// ---------------------------------------------------------------- norm (norm.cu)
struct NormArgs {
    int dtype;
    int64_t rows;
    int D;
    const void *x; int64_t ld_x;
    const void *delta; int64_t ld_delta;   // nullptr: no addition
    const void *w;
    float eps;
    void *x_out; int64_t ld_xo;            // nullptr: not stored
    void *y; int64_t ld_y;                 // nullptr: not stored
    void *y8;                              // FP8 codes + exponents, or nullptr
};
hcsa_status launch_add_rmsnorm(const NormArgs &a, cudaStream_t st);

// ---------------------------------------------------------------- prefill
// fp32 storage of an fp32 result
__device__ __forceinline__ void store_val(float *p, float v) { *p = v; }

struct SwaArgs {
    int dtype;
    int T, H, Hkv, dh, window, sinks;
    float scale;
    const void *q; int64_t ld_q;
    const void *k; int64_t ld_k;
    const void *v; int64_t ld_v;
    void *out; int64_t ld_out;
    int row0, row1;                        // query rows computed
    int *status;
};
hcsa_status launch_swa(const SwaArgs &a, cudaStream_t st);        // chooses the kernel
hcsa_status launch_swa_simt(const SwaArgs &a, cudaStream_t st);
bool swa_tc_supported(const SwaArgs &a);                          // bf16, dh 64 or 128, a positive scale
hcsa_status launch_swa_tc(const SwaArgs &a, cudaStream_t st);
int sm_grid(int per_sm);                                      // SMs of the device x per_sm
// Opt in to `bytes` of dynamic shared memory, once per kernel (its own `done`) and device.
bool shared_opt_in(const void *kernel, int bytes, bool *done);

// Keys of a block of consecutive queries [t_first, t_last]: `pad` columns for the first tokens that lie
// outside the window of the block's first query (n_sink of them real), then one column per token from w0
// to t_last.  Column c holds token c (c < pad) or w0 + c - pad.
struct BlockKeys {
    int n_sink, pad, w0, n;
    __device__ __forceinline__ int token(int c) const { return c < pad ? c : w0 + c - pad; }
};
__device__ __forceinline__ BlockKeys block_keys(int t_first, int t_last, int window, int sinks, int granule) {
    BlockKeys b;
    b.w0 = t_first - window + 1 > 0 ? t_first - window + 1 : 0;
    b.n_sink = sinks < b.w0 ? sinks : b.w0;
    b.pad = (b.n_sink + granule - 1) / granule * granule;
    b.n = b.pad + t_last - b.w0 + 1;
    return b;
}
// Is column c of the block seen by query t?
__device__ __forceinline__ bool column_seen(const BlockKeys &b, int c, int t, int window, int sinks) {
    if (c < b.pad) return c < b.n_sink;
    const int j = b.w0 + c - b.pad;
    return j <= t && (j > t - window || j < sinks);
}

// ---------------------------------------------------------------- paged cache
struct PageArgs {
    int dtype;
    bool lowprec;
    int B, Hkv, dh, page, n_pages, max_pages;
    void *k_pages, *v_pages;
    const int32_t *table;
    int *status;
};
hcsa_status launch_page_append(const PageArgs &a, int64_t rows, const int32_t *pos, const int32_t *seq, const void *k,
                               int64_t ld_k, const void *v, int64_t ld_v, cudaStream_t st);

struct DecodeArgs {
    PageArgs c;
    int H, window, sinks;
    float scale;
    const int32_t *pos;
    const void *q; int64_t ld_q;
    void *out; int64_t ld_out;
    void *ws;
};
size_t swa_decode_ws_bytes(int dtype, int B, int dh);
hcsa_status launch_swa_decode(const DecodeArgs &a, cudaStream_t st);

// Chunks of CT tokens (aligned, and CT divides the page: a chunk never crosses one) that the new token of a
// sequence reads: those of the first tokens, then those from the window's first chunk on (from token 0 when
// the two meet).
template <int CT>
struct DecodeKeys {
    int pos, w0, n_far, far_end, n;        // far_end: token of chunk n_far (the window's first chunk)
    __device__ __forceinline__ int token(int c) const { return c < n_far ? CT * c : far_end + CT * (c - n_far); }
    __device__ __forceinline__ bool seen(int j, int sinks) const { return j <= pos && (j >= w0 || j < sinks); }
    // every token of the chunk that starts at j
    __device__ __forceinline__ bool all_seen(int j, int sinks) const {
        return j + CT - 1 <= pos && (j >= w0 || j + CT <= sinks);
    }
};
template <int CT>
__device__ __forceinline__ DecodeKeys<CT> decode_keys(int pos, int window, int sinks, int64_t capacity, int *status) {
    DecodeKeys<CT> k{pos, 0, 0, 0, 0};
    if (pos < 0) return k;
    if (pos >= capacity) {
        report(status, kStatusBounds);
        return k;
    }
    k.w0 = pos - window + 1 > 0 ? pos - window + 1 : 0;
    k.far_end = k.w0 / CT * CT;
    k.n_far = ((sinks < k.w0 ? sinks : k.w0) + CT - 1) / CT;
    if (CT * k.n_far >= k.far_end) k.n_far = k.far_end = 0;
    k.n = k.n_far + (pos - k.far_end) / CT + 1;
    return k;
}

// Exponent of a 32-channel block in the pages and the norm's output: the smallest e with
// amax / 2^e <= 448, held to [-126, 120] so that 2^e and 2^-e are ordinary floats.
__device__ __forceinline__ int page_exponent(float amax) {
    if (!(amax < INFINITY)) return 120;
    if (!(amax > 0.f)) return 0;
    // amax = m 2^k: k - 8, one more where the mantissa is above 1.75 (the sum carries into the exponent field)
    const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 135;
    return e < -126 ? -126 : e;
}
// 8 channels -> 8 codes of x / 2^e (e in [-126, 120]); one rounding.  At e = 120 a finite value above 248 2^120
// would round up to 2^128, which fp32 and bf16 hold as infinity: it takes the code 240 instead (within half a step).
__device__ __forceinline__ uint2 codes_of(const float *v, int e) {
    const float inv = lp::pow2f(-e);
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v[i] * inv;
    if (e == 120) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(t[i]) < INFINITY) t[i] = fminf(fmaxf(t[i], -240.f), 240.f);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(t[2 * i], t[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

}  // namespace hcsa
