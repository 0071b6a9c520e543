// Residual addition with root-mean-square norm: s = x + delta, x_out = round(s), y = s / sqrt(mean(s^2) + eps) w,
// y in the storage type and / or as block-scaled FP8.
//
// HBM-bound (about two operations per byte): each row is read once into registers (the raw vectors of x and
// delta), reduced, and written from registers.  A row belongs to `tpr` threads of a block (a power of two);
// several rows share a block when rows are short.
#include "sliding.cuh"

namespace hcsa {

namespace {

template <typename S>
struct Row {
    static constexpr int V = Traits<S>::VEC;
    static __device__ __forceinline__ void unpack(const uint4 &r, float *v) {
        const S *e = reinterpret_cast<const S *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)e[i];
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        uint4 r;
        S *e = reinterpret_cast<S *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) store_val(&e[i], v[i]);
        return r;
    }
};

// The sum of squares is fp32 (each thread's at most 32 values, then a tree); with an FP8 output it is fp64, so that
// a block maximum next to a power-of-two border can be placed on the right side of it.
template <typename S, int VPT, bool FP8>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(NormArgs a, int tpr) {
    using R = Row<S>;
    constexpr int V = R::V;
    using Sum = typename std::conditional<FP8, double, float>::type;
    __shared__ Sum red[32];
    const int tid = threadIdx.x & (tpr - 1), sub = threadIdx.x / tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + sub;
    const bool live = row < a.rows;
    const int nvec = a.D / V;
    const S *xr = (const S *)a.x + row * a.ld_x;
    const S *dr = (const S *)a.delta + row * a.ld_delta;
    uint4 x[VPT], d[VPT], w[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        x[i] = d[i] = w[i] = make_uint4(0, 0, 0, 0);
        if (live && c < nvec) {
            x[i] = *reinterpret_cast<const uint4 *>(xr + c * V);
            if (a.delta) d[i] = *reinterpret_cast<const uint4 *>(dr + c * V);
            w[i] = __ldg(reinterpret_cast<const uint4 *>((const S *)a.w + c * V));
        }
    }
    Sum sum = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        float xv[V], dv[V];
        R::unpack(x[i], xv);
        R::unpack(d[i], dv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const Sum s = (Sum)xv[e] + (Sum)dv[e];
            sum += s * s;
        }
        if (a.x_out) {
            const int c = tid + i * tpr;
            if (live && c < nvec) {
                float s[V];
#pragma unroll
                for (int e = 0; e < V; ++e) s[e] = xv[e] + dv[e];
                *reinterpret_cast<uint4 *>((S *)a.x_out + row * a.ld_xo + c * V) = R::pack(s);
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < tpr) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (tpr > 32) {   // uniform: every thread of the block takes part
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0;
        for (int i = 0; i < (tpr >> 5); ++i) sum += red[sub * (tpr >> 5) + i];   // same order in every thread
    }
    if (!live) return;
    const Sum ms = sum / (Sum)a.D + (Sum)a.eps;
    const Sum rstd_w = (Sum)1 / sqrt(ms);
    const float rstd = (float)rstd_w;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        if (c >= nvec) break;
        float xv[V], dv[V], wv[V], y[V];
        R::unpack(x[i], xv);
        R::unpack(d[i], dv);
        R::unpack(w[i], wv);
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = (xv[e] + dv[e]) * rstd * wv[e];
        if (a.y) *reinterpret_cast<uint4 *>((S *)a.y + row * a.ld_y + c * V) = R::pack(y);
        if constexpr (FP8) {
            const float amax = lp::block_amax(y);
            int e = page_exponent(amax);
            // y is four roundings away from the exact value: within 2^-20 of the border 1.75 2^k the block's
            // maximum is taken in fp64
            const float f = amax * lp::pow2f(-e);   // (224, 448] unless held or zero
            if (fabsf(f - 448.f) < 448.f * 0x1p-20f || fabsf(f - 224.f) < 224.f * 0x1p-20f) {
                double big = 0;
#pragma unroll
                for (int q = 0; q < V; ++q)
                    big = fmax(big, fabs(((double)xv[q] + (double)dv[q]) * rstd_w * (double)wv[q]));
                const unsigned grp = 0xFu << (threadIdx.x & 28);
                big = fmax(big, __shfl_xor_sync(grp, big, 1));
                big = fmax(big, __shfl_xor_sync(grp, big, 2));
                const double at = ldexp(448.0, e);
                e = big > at ? e + 1 : (big <= 0.5 * at && e > -126) ? e - 1 : e;
            }
            uint8_t *codes = (uint8_t *)a.y8;
            *reinterpret_cast<uint2 *>(codes + row * a.D + c * V) = codes_of(y, e);
            if ((c & 3) == 0) ((int8_t *)codes)[a.rows * a.D + row * (a.D / 32) + c / 4] = (int8_t)e;
        }
    }
}

template <typename S, int VPT, bool FP8>
void launch(const NormArgs &a, int tpr, cudaStream_t st) {
    const int threads = tpr > 256 ? tpr : 256, per = threads / tpr;
    add_rmsnorm_kernel<S, VPT, FP8><<<(unsigned)((a.rows + per - 1) / per), threads, 0, st>>>(a, tpr);
}
template <typename S, bool FP8>
void launch_v(const NormArgs &a, int vpt, int tpr, cudaStream_t st) {
    if (vpt == 1) launch<S, 1, FP8>(a, tpr, st);
    else if (vpt == 2) launch<S, 2, FP8>(a, tpr, st);
    else launch<S, 4, FP8>(a, tpr, st);
}

}  // namespace

hcsa_status launch_add_rmsnorm(const NormArgs &a, cudaStream_t st) {
    if (a.rows == 0) return HCSA_OK;
    const int nvec = a.D / (a.dtype == HCSA_BF16 ? 8 : 4);
    // few rows: one vector per thread (shortest path); many: four (fewer threads to reduce over, more bytes in flight)
    int vpt = a.rows <= 1024 ? 1 : 4;
    while (vpt < 4 && (nvec + vpt - 1) / vpt > 1024) vpt *= 2;
    int tpr = 32;
    while (tpr < (nvec + vpt - 1) / vpt) tpr *= 2;
    if (a.dtype == HCSA_F32) launch_v<float, false>(a, vpt, tpr, st);
    else if (a.y8) launch_v<__nv_bfloat16, true>(a, vpt, tpr, st);
    else launch_v<__nv_bfloat16, false>(a, vpt, tpr, st);
    count_launch();
    return check_launch();
}

}  // namespace hcsa
