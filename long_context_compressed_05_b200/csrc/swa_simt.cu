// Sliding-window prefill attention on the CUDA cores: fp32 storage, and bf16 head dims the tensor-core kernel does
// not take.  Flash-style: a block owns BM consecutive (token, head of the group) rows of one key head and walks
// the keys its tokens see in tiles of BN, all operands in shared memory as fp32, online softmax.
//
// 256 threads as 16 x 16: thread (ty, tx) owns rows ty RM .. and key columns tx + 16 j of a score tile, and
// dims 4 tx + 64 j of the output rows.  Bound by the FP32 pipe and shared-memory reads (each 16-byte read feeds
// eight FMAs at BM = 64, BN = 32).
#include "sliding.cuh"

namespace hcsa {

namespace {

template <typename S, int DH, int BM, int BN>
struct SimtSmem {
    float q[BM][DH + 4], k[BN][DH + 4], v[BN][DH], p[BM][BN + 4];
    int bad[BM];
};

template <typename S, int DH, int BM, int BN>
__global__ void __launch_bounds__(256) swa_simt_kernel(SwaArgs a, int64_t blocks_per_head) {
    constexpr int V = Traits<S>::VEC, RM = BM / 16, RN = BN / 16, DN = DH / 64;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SimtSmem<S, DH, BM, BN> &sm = *reinterpret_cast<SimtSmem<S, DH, BM, BN> *>(smem_raw);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int G = a.H / a.Hkv;
    const int g = (int)(blockIdx.x / blocks_per_head);
    // latest tokens (the most keys) first
    const int64_t r0 = (int64_t)a.row0 * G + (blocks_per_head - 1 - blockIdx.x % blocks_per_head) * BM;
    const int64_t r_end = (int64_t)a.row1 * G;
    const int64_t r_last = (r0 + BM < r_end ? r0 + BM : r_end) - 1;
    const BlockKeys bk = block_keys((int)(r0 / G), (int)(r_last / G), a.window, a.sinks, 1);
    const float scale = a.scale * 1.4426950408889634f;

    auto load_rows = [&](auto &dst, int rows, auto src_of) {   // src_of(row): pointer or nullptr (zeros)
        for (int i = threadIdx.x; i < rows * (DH / V); i += 256) {
            const int r = i / (DH / V), c = (i % (DH / V)) * V;
            const S *src = src_of(r);
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = 0.f;
            if (src && c < a.dh) {
                const uint4 raw = __ldg(reinterpret_cast<const uint4 *>(src + c));
                const S *e8 = reinterpret_cast<const S *>(&raw);
#pragma unroll
                for (int e = 0; e < V; ++e) f[e] = (float)e8[e];
            }
#pragma unroll
            for (int e = 0; e < V; e += 4)
                *reinterpret_cast<float4 *>(&dst[r][c + e]) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
    };
    load_rows(sm.q, BM, [&](int r) -> const S * {
        const int64_t row = r0 + r;
        if (row > r_last) return nullptr;
        return (const S *)a.q + (row / G) * a.ld_q + (int64_t)(g * G + (int)(row % G)) * a.dh;
    });

    float o[RM][DN][4], m[RM], l[RM];
    int tok[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        const int64_t row = r0 + ty * RM + i;
        tok[i] = row <= r_last ? (int)(row / G) : -1;
#pragma unroll
        for (int j = 0; j < DN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    }
    // K and V of the next tile wait in registers while this one is worked on
    constexpr int NL = BN * (DH / V) / 256;
    static_assert(BN * (DH / V) % 256 == 0, "whole vectors per thread");
    uint4 kr[NL], vr[NL];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = j * 256 + threadIdx.x, c = c0 + i / (DH / V), d = (i % (DH / V)) * V;
            kr[j] = vr[j] = make_uint4(0, 0, 0, 0);
            if (c < bk.n && d < a.dh) {
                const int64_t t = bk.token(c);
                kr[j] = __ldg(reinterpret_cast<const uint4 *>((const S *)a.k + t * a.ld_k + (int64_t)g * a.dh + d));
                vr[j] = __ldg(reinterpret_cast<const uint4 *>((const S *)a.v + t * a.ld_v + (int64_t)g * a.dh + d));
            }
        }
    };
    auto widen = [](const uint4 &raw, float *dst) {
        const S *e8 = reinterpret_cast<const S *>(&raw);
#pragma unroll
        for (int e = 0; e < V; e += 4)
            *reinterpret_cast<float4 *>(dst + e) =
                make_float4((float)e8[e], (float)e8[e + 1], (float)e8[e + 2], (float)e8[e + 3]);
    };
    fetch(0);
    for (int c0 = 0; c0 < bk.n; c0 += BN) {
        __syncthreads();   // the previous tile's readers are done
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = j * 256 + threadIdx.x, r = i / (DH / V), d = (i % (DH / V)) * V;
            widen(kr[j], &sm.k[r][d]);
            widen(vr[j], &sm.v[r][d]);
        }
        if (c0 + BN < bk.n) fetch(c0 + BN);
        __syncthreads();
        float s[RM][RN];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < RN; ++j) s[i][j] = 0.f;
#pragma unroll 4
        for (int d = 0; d < DH; d += 4) {
            float4 kq[RN];
#pragma unroll
            for (int j = 0; j < RN; ++j) kq[j] = *reinterpret_cast<const float4 *>(&sm.k[tx + 16 * j][d]);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[ty * RM + i][d]);
#pragma unroll
                for (int j = 0; j < RN; ++j)
                    s[i][j] += qv.x * kq[j].x + qv.y * kq[j].y + qv.z * kq[j].z + qv.w * kq[j].w;
            }
        }
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            float mt = m[i];
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                const int c = c0 + tx + 16 * j;
                const bool seen = c < bk.n && column_seen(bk, c, tok[i], a.window, a.sinks);
                s[i][j] = seen ? s[i][j] * scale : -INFINITY;
                mt = fmaxf(mt, s[i][j]);
            }
#pragma unroll
            for (int q = 8; q; q >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, q));
            const float ref = mt == -INFINITY ? 0.f : mt;   // a row that has seen no key yet: every weight 0
            const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - ref);
            m[i] = mt;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                const float p = exp2f(s[i][j] - ref);
                sum += p;
                sm.p[ty * RM + i][tx + 16 * j] = p;
            }
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int j = 0; j < DN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] *= f;
        }
        __syncwarp();   // a row's 16 threads are in one warp
#pragma unroll 2
        for (int c = 0; c < BN; c += 4) {
            float4 p[RM];
#pragma unroll
            for (int i = 0; i < RM; ++i) p[i] = *reinterpret_cast<const float4 *>(&sm.p[ty * RM + i][c]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < DN; ++j) {
                    const float4 vv = *reinterpret_cast<const float4 *>(&sm.v[c + e][4 * tx + 64 * j]);
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        const float w = e == 0 ? p[i].x : e == 1 ? p[i].y : e == 2 ? p[i].z : p[i].w;
                        o[i][j][0] += w * vv.x;
                        o[i][j][1] += w * vv.y;
                        o[i][j][2] += w * vv.z;
                        o[i][j][3] += w * vv.w;
                    }
                }
        }
    }
    if (threadIdx.x < BM) sm.bad[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RM; ++i) {
#pragma unroll
        for (int q = 8; q; q >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], q);
        if (tok[i] < 0) continue;
        const int64_t row = r0 + ty * RM + i;
        S *dst = (S *)a.out + (int64_t)tok[i] * a.ld_out + (int64_t)(g * G + (int)(row % G)) * a.dh;
        bool fine = true;
#pragma unroll
        for (int j = 0; j < DN; ++j) {
            const int d = 4 * tx + 64 * j;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = o[i][j][e] / l[i];
                fine = fine && (d + e >= a.dh || fabsf(y) < INFINITY);
                if (d + e < a.dh) store_val(dst + d + e, y);
            }
        }
        if (!fine) sm.bad[ty * RM + i] = 1;
    }
    __syncthreads();
    const int t_last = (int)(r_last / G), lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < BM; r += 8) {
        if (!sm.bad[r]) continue;
        const int t = (int)((r0 + r) / G);
        const int h = g * G + (int)((r0 + r) % G);
        if ((values_bad<S>(a, g, bk.w0, (int64_t)t - a.window + 1, lane) || values_bad<S>(a, g, t + 1, t_last + 1, lane)) &&
            !row_explained<S>(a, t, h, lane, 0, a.dh))
            attend_row<S>(a, t, h, lane, 0, a.dh);
    }
}

template <typename S, int DH, int BM, int BN>
hcsa_status launch(const SwaArgs &a, cudaStream_t st) {
    constexpr int smem = (int)sizeof(SimtSmem<S, DH, BM, BN>);
    static_assert(smem <= 232448, "shared memory per CTA");
    static bool opted[64];
    if (!shared_opt_in((const void *)swa_simt_kernel<S, DH, BM, BN>, smem, opted)) return HCSA_ERR_CUDA;
    const int64_t per = ((int64_t)(a.row1 - a.row0) * (a.H / a.Hkv) + BM - 1) / BM;
    if (per * a.Hkv > INT32_MAX) return HCSA_ERR_UNSUPPORTED;
    swa_simt_kernel<S, DH, BM, BN><<<(unsigned)(per * a.Hkv), 256, smem, st>>>(a, per);
    count_launch();
    return check_launch();
}

template <typename S>
hcsa_status launch_dh(const SwaArgs &a, cudaStream_t st) {
    if (a.dh <= 64) return launch<S, 64, 64, 32>(a, st);
    if (a.dh <= 128) return launch<S, 128, 64, 32>(a, st);
    if (a.dh <= 256) return launch<S, 256, 64, 32>(a, st);
    return launch<S, 512, 32, 16>(a, st);
}

}  // namespace

hcsa_status launch_swa_simt(const SwaArgs &a, cudaStream_t st) {
    return a.dtype == HCSA_F32 ? launch_dh<float>(a, st) : launch_dh<__nv_bfloat16>(a, st);
}

hcsa_status launch_swa(const SwaArgs &a, cudaStream_t st) {
    return swa_tc_supported(a) ? launch_swa_tc(a, st) : launch_swa_simt(a, st);
}

}  // namespace hcsa
