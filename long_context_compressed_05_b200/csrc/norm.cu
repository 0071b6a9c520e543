// Residual addition with root-mean-square norm: s = x + delta, x_out = round(s), y = s / sqrt(mean(s^2) + eps) w,
// y in the storage type and / or as block-scaled FP8.
//
// HBM-bound (about two operations per byte): each row is read once into registers, reduced, and written from
// registers.  A row belongs to `tpr` threads of a block (a power of two);
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

// Sum over the row's tpr threads, in the same order in all of them; every thread of the block calls it.
template <typename T>
__device__ __forceinline__ T row_sum(T v, int tpr, int sub, T *red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr > 32) {
        __syncthreads();             // red may still be read
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0;
        for (int i = 0; i < (tpr >> 5); ++i) v += red[sub * (tpr >> 5) + i];
    }
    return v;
}

// The sum of squares is fp32: a thread's at most 32 values (in eight partial sums), then a tree of at most 10: y is
// within 2^-19 of its exact value.  FP8: a block whose maximum lies within 2^-18 of a power-of-two border makes its
// row sum once more in fp64 and takes the border's side from that; one row in a thousand has such a block.  (131072 rows
// of 2048 took 833 us with every sum in fp64 and 427 when that went; later steps brought it to 315.)
// The row's 1 / sqrt(mean + eps) in fp64, read again (out of line: it would double the kernel's registers).
template <typename S>
__device__ __noinline__ double exact_rstd(const NormArgs &a, int64_t row, bool live, int tid, int tpr, int sub, double *red) {
    constexpr int V = Traits<S>::VEC;
    double sum = 0;
    for (int c = tid * V; live && c < a.D; c += tpr * V)
        for (int e = c; e < c + V; ++e) {
            const double s = (double)((const S *)a.x)[row * a.ld_x + e] +
                             (a.delta ? (double)((const S *)a.delta)[row * a.ld_delta + e] : 0.0);
            sum += s * s;
        }
    return 1 / sqrt(row_sum(sum, tpr, sub, red) / a.D + (double)a.eps);
}
// A block's maximum in fp32, over its four lanes of `lanes`; NaN only where all 32 values are.
__device__ __forceinline__ float row_block_amax(const float *v, unsigned lanes) {
    float a = fmaxf(fabsf(v[0]), fabsf(v[1]));
#pragma unroll
    for (int i = 2; i < 8; i += 2) a = fmaxf(a, fmaxf(fabsf(v[i]), fabsf(v[i + 1])));
    a = fmaxf(a, __shfl_xor_sync(lanes, a, 1));
    return fmaxf(a, __shfl_xor_sync(lanes, a, 2));
}
// Does the exponent e of a block hang on the last bits of its maximum?  amax / 2^e lies in (224, 448] unless e is held,
// or the block has no finite value but zero: those have nothing to decide.
__device__ __forceinline__ bool at_border(float amax, int e) {
    const float f = amax * lp::pow2f(-e);
    return fabsf(f - 448.f) < 448.f * 0x1p-18f || fabsf(f - 224.f) < 224.f * 0x1p-18f;
}
// The exponents of the row's blocks at a border once more from the maxima in fp64, and the codes where the exponent
// changes; each thread reads its own vectors of x and delta again.
template <typename S>
__device__ __noinline__ void exact_blocks(const NormArgs &a, int64_t row, bool live, int tid, int tpr, int sub, float rstd,
                                          double *red) {
    constexpr int V = Traits<S>::VEC;
    const double exact = exact_rstd<S>(a, row, live, tid, tpr, sub, red);
    uint8_t *codes = (uint8_t *)a.y8 + row * a.D;
    int8_t *exps = (int8_t *)a.y8 + a.rows * a.D + row * (a.D / 32);
    for (int c = tid * V; live && c < a.D; c += tpr * V) {   // the four lanes of a block stay together
        double big = 0;
        float y[V];
        for (int q = 0; q < V; ++q) {
            const float x = (float)((const S *)a.x)[row * a.ld_x + c + q];
            const float d = a.delta ? (float)((const S *)a.delta)[row * a.ld_delta + c + q] : 0.f;
            const float w = (float)((const S *)a.w)[c + q];
            big = fmax(big, fabs(((double)x + (double)d) * exact * (double)w));
            y[q] = (x + d) * rstd * w;
        }
        const unsigned grp = 0xFu << (threadIdx.x & 28);
        big = fmax(big, __shfl_xor_sync(grp, big, 1));
        big = fmax(big, __shfl_xor_sync(grp, big, 2));
        const float amax = row_block_amax(y, grp);
        const int was = page_exponent(amax);
        if (!at_border(amax, was)) continue;
        const double at = ldexp(448.0, was);   // the fp32 exponent is right or one off
        const int e = big > at && was < 120 ? was + 1 : big <= 0.5 * at && was > -126 ? was - 1 : was;
        if (e == was) continue;
        *reinterpret_cast<uint2 *>(codes + c) = codes_of(y, e);
        if ((c & 31) == 0) exps[c / 32] = (int8_t)e;
    }
}

template <typename S, int VPT, bool FP8>
__global__ void __launch_bounds__(1024) add_rmsnorm_kernel(NormArgs a, int tpr) {
    using R = Row<S>;
    constexpr int V = R::V;
    __shared__ float red[32];
    __shared__ double redd[FP8 ? 32 : 1];
    const int tid = threadIdx.x & (tpr - 1), sub = threadIdx.x / tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + sub;
    const bool live = row < a.rows;
    const int nvec = a.D / V;
    const S *xr = (const S *)a.x + row * a.ld_x;
    const S *dr = (const S *)a.delta + row * a.ld_delta;
    uint4 x[VPT], d[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        x[i] = d[i] = make_uint4(0, 0, 0, 0);
        if (live && c < nvec) {
            x[i] = *reinterpret_cast<const uint4 *>(xr + c * V);
            if (a.delta) d[i] = *reinterpret_cast<const uint4 *>(dr + c * V);
        }
    }
    // FP8 with x_out = x (or delta): stored last, from a second reading, since the exact path reads them again
    const bool in_place = FP8 && a.x_out && (a.x_out == a.x || a.x_out == a.delta);
    float v[VPT][V], part[V];
#pragma unroll
    for (int e = 0; e < V; ++e) part[e] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        float dv[V];
        R::unpack(x[i], v[i]);
        R::unpack(d[i], dv);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[i][e] += dv[e];
            part[e] += v[i][e] * v[i][e];
        }
        if (a.x_out && !in_place && live && c < nvec)
            *reinterpret_cast<uint4 *>((S *)a.x_out + row * a.ld_xo + c * V) = R::pack(v[i]);
    }
#pragma unroll
    for (int w = V / 2; w; w >>= 1)
#pragma unroll
        for (int e = 0; e < w; ++e) part[e] += part[e + w];
    const float rstd = 1.f / sqrtf(row_sum(part[0], tpr, sub, red) / (float)a.D + a.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = tid + i * tpr;
        if (c < nvec) {
            float wv[V];
            R::unpack(__ldg(reinterpret_cast<const uint4 *>((const S *)a.w + c * V)), wv);
#pragma unroll
            for (int e = 0; e < V; ++e) v[i][e] = v[i][e] * rstd * wv[e];
            if (a.y && live) *reinterpret_cast<uint4 *>((S *)a.y + row * a.ld_y + c * V) = R::pack(v[i]);
        }
    }
    if constexpr (FP8) {
        unsigned near = 0;
        uint8_t *codes = (uint8_t *)a.y8;
        int8_t *exps = (int8_t *)codes + a.rows * a.D;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {   // D % 32 == 0: the four lanes of a block are in or out together
            const int c = tid + i * tpr;
            const float amax = row_block_amax(v[i], 0xffffffffu);   // (a partial mask would cost a synchronisation per shuffle)
            const int e = page_exponent(amax);
            near |= at_border(amax, e);
            if (live && c < nvec) {
                *reinterpret_cast<uint2 *>(codes + row * a.D + c * V) = codes_of(v[i], e);
                if ((c & 3) == 0) exps[row * (a.D / 32) + c / 4] = (int8_t)e;
            }
        }
        if (tpr > 32 ? __syncthreads_or(near) : __any_sync(0xffffffffu, near))
            exact_blocks<S>(a, row, live, tid, tpr, sub, rstd, redd);
        if (in_place && live)
            for (int c = tid; c < nvec; c += tpr) {
                float xv[V], dv[V];
                R::unpack(*reinterpret_cast<const uint4 *>(xr + c * V), xv);
                R::unpack(a.delta ? *reinterpret_cast<const uint4 *>(dr + c * V) : make_uint4(0, 0, 0, 0), dv);
#pragma unroll
                for (int e = 0; e < V; ++e) xv[e] += dv[e];
                *reinterpret_cast<uint4 *>((S *)a.x_out + row * a.ld_xo + c * V) = R::pack(xv);
            }
    }
}

template <typename S, int VPT, bool FP8>
void launch(const NormArgs &a, int tpr, cudaStream_t st) {
    const int threads = tpr > 128 ? tpr : 128, per = threads / tpr;
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
    // few rows: one vector per thread (the shortest path); many: up to four (131072 rows of 2048, FP8, in a captured graph:
    // 315 us; 424 with two, more threads to reduce over; 662 with eight, fewer warps per SM)
    int vpt = 1;
    while (vpt < 4 && ((a.rows > 1024 && vpt * 32 < nvec) || vpt * 1024 < nvec)) vpt *= 2;
    int tpr = 32;
    while (tpr < (nvec + vpt - 1) / vpt) tpr *= 2;
    if (a.dtype == HCSA_F32) launch_v<float, false>(a, vpt, tpr, st);
    else if (a.y8) launch_v<__nv_bfloat16, true>(a, vpt, tpr, st);
    else launch_v<__nv_bfloat16, false>(a, vpt, tpr, st);
    count_launch();
    return check_launch();
}

}  // namespace hcsa
