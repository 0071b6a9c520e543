// Sliding-window prefill attention on the CUDA cores: fp32 storage, and bf16 head dims the tensor-core kernel does
// not take.  Flash-style: a block owns BM consecutive (token, head of the group) rows of one key head and walks
// the keys its tokens see in tiles of BN, all operands in shared memory as fp32, online softmax.
//
// A group of 128 threads as 16 x 8: thread (ty, tx) owns rows ty + 16 i, key columns tx + 8 j of a score tile, and dims
// 4 tx + 32 j of the output rows.  A warp is then 4 rows x 8 columns, whose 16-byte reads touch each bank once, and RM =
// RN = 4 make 64 FMAs of eight reads.  Up to dh 64 a block has two groups, which take every other tile of keys and are
// joined at the end: a short window over a few thousand tokens has too few blocks to hide the reads' latency otherwise
// (2048 tokens, 8 heads of 64, window 128: 45.4 us, 48.8 with one group).  Bound by issue of FMAs between reads (4096
// tokens, 16 heads over 4 of 128, window 1000: 912 us, 43% of the FP32 rate; 1143 as 256 threads of 16 x 16 with 32 FMAs of
// six reads).  bf16 with the head dims that come here, causal 4096 tokens, 16 heads over 4: 2.45 ms at dh 72, 5.0 ms at
// dh 256.  fp32 above dh 128 spills registers (268 bytes up to dh 256, 204 up to 512), as no smaller tile was tried there.
#include "sliding.cuh"

namespace hcsa {

namespace {

constexpr int kThreads = 128;       // of a group
template <int DH> constexpr int groups_of() { return DH <= 64 ? 2 : 1; }

template <typename S, int DH, int BM, int BN>
struct SimtSmem {
    struct Tile {
        float k[BN][DH + 4], v[BN][DH], p[BM][BN + 4];
    };
    float q[BM][DH + 4];
    Tile t[groups_of<DH>()];
};

template <typename S, int DH, int BM, int BN>
__global__ void __launch_bounds__(kThreads * groups_of<DH>(), DH <= 64 ? 2 : DH <= 128 ? 3 : 1) swa_simt_kernel(SwaArgs a, int64_t blocks_per_head) {
    constexpr int V = Traits<S>::VEC, RM = BM / 16, RN = BN / 8, DN = DH / 32;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SimtSmem<S, DH, BM, BN> &sm = *reinterpret_cast<SimtSmem<S, DH, BM, BN> *>(smem_raw);
    constexpr int NG = groups_of<DH>();
    const int tid = threadIdx.x % kThreads, group = threadIdx.x / kThreads;
    typename SimtSmem<S, DH, BM, BN>::Tile &tile = sm.t[group];
    const int tx = tid & 7, ty = tid >> 3;
    auto sync_group = [&]() {
        if (NG == 1) __syncthreads();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kThreads) : "memory");
    };
    const int G = a.H / a.Hkv;
    const int g = (int)(blockIdx.x / blocks_per_head);
    // latest tokens (the most keys) first
    const int64_t r0 = (int64_t)a.row0 * G + (blocks_per_head - 1 - blockIdx.x % blocks_per_head) * BM;
    const int64_t r_end = (int64_t)a.row1 * G;
    const int64_t r_last = (r0 + BM < r_end ? r0 + BM : r_end) - 1;
    // row r of the block: token t_first + (rem + r) / G, head (rem + r) % G of the group
    const int t_first = (int)(r0 / G), t_end = (int)(r_last / G), rem = (int)(r0 % G), n_rows = (int)(r_last - r0) + 1;
    const BlockKeys bk = block_keys(t_first, t_end, a.window, a.sinks, 1);
    const float scale = a.scale * 1.4426950408889634f;

    auto load_rows = [&](auto &dst, int rows, auto src_of) {   // src_of(row): pointer or nullptr (zeros)
        for (int i = threadIdx.x; i < rows * (DH / V); i += kThreads * NG) {
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
        if (r >= n_rows) return nullptr;
        const int x = rem + r, t = x / G;
        return (const S *)a.q + (int64_t)(t_first + t) * a.ld_q + (int64_t)(g * G + x - t * G) * a.dh;
    });

    int tok[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) tok[i] = ty + 16 * i < n_rows ? t_first + (rem + ty + 16 * i) / G : -1;
    // K and V of the next tile wait in registers while this one is worked on
    constexpr int NL = BN * (DH / V) / kThreads;
    static_assert(BN * (DH / V) % kThreads == 0, "whole vectors per thread");
    constexpr bool kAhead = NL <= 4;   // else there are no registers for it
    uint4 kr[NL], vr[NL];
    auto fetch = [&](int c0) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = j * kThreads + tid, c = c0 + i / (DH / V), d = (i % (DH / V)) * V;
            kr[j] = vr[j] = make_uint4(0, 0, 0, 0);
            if (c < bk.n && d < a.dh) {
                const int64_t t = bk.token(c);
                kr[j] = __ldg(reinterpret_cast<const uint4 *>((const S *)a.k + t * a.ld_k + (int64_t)g * a.dh + d));
                vr[j] = __ldg(reinterpret_cast<const uint4 *>((const S *)a.v + t * a.ld_v + (int64_t)g * a.dh + d));
            }
        }
    };
    auto widen = [](const uint4 &raw, float *dst, bool finite) {
        const S *e8 = reinterpret_cast<const S *>(&raw);
        float f[V];
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = (float)e8[e];
        if (finite) {
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = fabsf(f[e]) < INFINITY ? f[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < V; e += 4) *reinterpret_cast<float4 *>(dst + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    };
    // Every masked key has the weight 0, and 0 times an infinite or NaN value is NaN.  So a block with a row that came
    // out non-finite is computed a second time without such values, which then reach the rows that see them
    for (int again = 0;; again = 1) {
    float o[RM][DN][4], m[RM], l[RM];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < DN; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
    }
    if (kAhead) fetch(group * BN);
    __syncthreads();       // Q, or the first pass's last readers
    for (int c0 = group * BN; c0 < bk.n; c0 += NG * BN) {
        sync_group();      // the previous tile's readers are done
        if (!kAhead) fetch(c0);
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = j * kThreads + tid, r = i / (DH / V), d = (i % (DH / V)) * V;
            widen(kr[j], &tile.k[r][d], false);
            widen(vr[j], &tile.v[r][d], again);
        }
        if (kAhead && c0 + NG * BN < bk.n) fetch(c0 + NG * BN);
        sync_group();
        // every column seen by every row?
        const bool clean = c0 >= bk.pad && bk.token(c0 + BN - 1) <= t_first && bk.token(c0) > t_end - a.window;
        float s[RM][RN];
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < RN; ++j) s[i][j] = 0.f;
#pragma unroll 2
        for (int d = 0; d < DH; d += 4) {
            float4 kq[RN];
#pragma unroll
            for (int j = 0; j < RN; ++j) kq[j] = *reinterpret_cast<const float4 *>(&tile.k[tx + 8 * j][d]);
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const float4 qv = *reinterpret_cast<const float4 *>(&sm.q[ty + 16 * i][d]);
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
                const int c = c0 + tx + 8 * j;
                const bool seen = clean || (c < bk.n && column_seen(bk, c, tok[i], a.window, a.sinks));
                s[i][j] = seen ? s[i][j] * scale : -INFINITY;
                mt = fmaxf(mt, s[i][j]);
            }
#pragma unroll
            for (int q = 4; q; q >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, q));
            const float ref = mt == -INFINITY ? 0.f : mt;   // a row that has seen no key yet: every weight 0
            const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - ref);
            m[i] = mt;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < RN; ++j) {
                const float p = exp2f(s[i][j] - ref);
                sum += p;
                tile.p[ty + 16 * i][tx + 8 * j] = p;
            }
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int j = 0; j < DN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][j][e] *= f;
        }
        __syncwarp();   // a row's 8 threads are in one warp
#pragma unroll 2
        for (int c = 0; c < BN; c += 4) {
            float4 p[RM];
#pragma unroll
            for (int i = 0; i < RM; ++i) p[i] = *reinterpret_cast<const float4 *>(&tile.p[ty + 16 * i][c]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int j = 0; j < DN; ++j) {
                    const float4 vv = *reinterpret_cast<const float4 *>(&tile.v[c + e][4 * tx + 32 * j]);
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
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int q = 4; q; q >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], q);
    __syncthreads();
    if constexpr (NG == 2) {   // the second group's rows through its tile's memory
        float *x = reinterpret_cast<float *>(&sm.t[1]) + tid;
        constexpr int kEach = 2 + 4 * DN;
        static_assert(RM * kEach * kThreads * sizeof(float) <= sizeof(sm.t[1]), "the join fits");
        if (group == 1) {
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                x[(i * kEach) * kThreads] = m[i];
                x[(i * kEach + 1) * kThreads] = l[i];
#pragma unroll
                for (int j = 0; j < 4 * DN; ++j) x[(i * kEach + 2 + j) * kThreads] = o[i][j / 4][j % 4];
            }
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int i = 0; i < RM; ++i) {
                const float m1 = x[(i * kEach) * kThreads], l1 = x[(i * kEach + 1) * kThreads], mm = fmaxf(m[i], m1);
                const float ref = mm == -INFINITY ? 0.f : mm;
                const float f0 = m[i] == -INFINITY ? 0.f : exp2f(m[i] - ref), f1 = m1 == -INFINITY ? 0.f : exp2f(m1 - ref);
                l[i] = l[i] * f0 + l1 * f1;
#pragma unroll
                for (int j = 0; j < 4 * DN; ++j)
                    o[i][j / 4][j % 4] = o[i][j / 4][j % 4] * f0 + x[(i * kEach + 2 + j) * kThreads] * f1;
            }
        }
    }
    bool fine = true;
    auto row = [&](int i) { return (S *)a.out + (int64_t)tok[i] * a.ld_out + (int64_t)(g * G + (rem + ty + 16 * i) % G) * a.dh; };
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        if (tok[i] < 0 || group) continue;
        S *dst = row(i);
#pragma unroll
        for (int j = 0; j < DN; ++j) {
            const int d = 4 * tx + 32 * j;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float y = o[i][j][e] / l[i];
                fine = fine && (d + e >= a.dh || fabsf(y) < INFINITY);
                if (d + e < a.dh) store_val(dst + d + e, y);
            }
        }
    }
    if (again) {
        // infinite values that each row sees, by sign (NaN: both), a bit per channel: one sign makes the channel infinite, both
        // NaN; a row whose weights are NaN stays so
        using Bits = uint64_t;
        static_assert(4 * DN <= 64, "a bit per channel");
        Bits up[RM], down[RM];
#pragma unroll
        for (int i = 0; i < RM; ++i) up[i] = down[i] = 0;
        for (int c = 0; c < bk.n && !group; ++c) {
            const S *v = (const S *)a.v + (int64_t)bk.token(c) * a.ld_v + (int64_t)g * a.dh;
            Bits u = 0, w = 0;
#pragma unroll
            for (int j = 0; j < 4 * DN; ++j) {
                const int d = 4 * tx + 32 * (j / 4) + j % 4;
                const float f = d < a.dh ? (float)v[d] : 0.f;
                const Bits bit = fabsf(f) < INFINITY ? 0 : (Bits)1 << j;
                if (!(f < 0.f)) u |= bit;
                if (!(f > 0.f)) w |= bit;
            }
            if (!(u | w)) continue;
#pragma unroll
            for (int i = 0; i < RM; ++i)
                if (column_seen(bk, c, tok[i], a.window, a.sinks)) {
                    up[i] |= u;
                    down[i] |= w;
                }
        }
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            if (tok[i] < 0 || group || !(l[i] > 0.f)) continue;
            for (Bits any = up[i] | down[i]; any; any &= any - 1) {
                const int j = __ffsll(any) - 1;
                const bool u = up[i] >> j & 1, w = down[i] >> j & 1;
                store_val(row(i) + 4 * tx + 32 * (j / 4) + j % 4, u && w ? NAN : u ? INFINITY : -INFINITY);
            }
        }
    }
    if (again || !__syncthreads_or(!fine)) break;
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
    swa_simt_kernel<S, DH, BM, BN><<<(unsigned)(per * a.Hkv), kThreads * groups_of<DH>(), smem, st>>>(a, per);
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
