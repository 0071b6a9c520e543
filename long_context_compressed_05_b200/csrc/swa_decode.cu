// One-token attention over the paged cache: the split over CTAs, the joining kernel, and the CUDA-core kernel (fp32
// pages, and head dims the tensor-core kernel does not take).
//
// CUDA-core kernel: eight warps take the chunks of a segment in turn; within a chunk a warp takes four tokens
// at a time.  Each lane holds DH / 32 dims of the rows and of the query heads; the 4 x HB partial products are
// summed over lanes by a halving exchange (one shuffle per value), the weights go back by shuffles.  Groups
// of more than HB heads are separate units that read the rows again (from L2).  Loads go straight from global
// memory to registers, 16 bytes a lane, four rows of K and of V at a time.  32 sequences up to 8192 tokens, 64 heads over 8,
// in a captured graph: fp32 pages of dh 128 402 us (2745 GB/s), bf16 pages of dh 96 601 us (688 GB/s); bound by the FMAs and
// shuffles of a row.
#include "decode_split.cuh"

namespace hcsa {

namespace {

constexpr int kWarps = 8;
constexpr int kPerSM = 2;            // CTAs per SM of a split step

template <int DH> constexpr int heads_of() { return DH <= 256 ? 8 : 2; }

// DH / 32 dims of one cache row
template <typename S, bool FP8, int DH>
__device__ __forceinline__ void load_row(const DecodeArgs &a, const void *pages, int64_t line, int lane, float *f) {
    constexpr int N = DH / 32;
    const int d0 = lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = 0.f;
    if constexpr (FP8) {
        const uint8_t *codes = (const uint8_t *)pages;
        const int64_t lines = (int64_t)a.c.n_pages * a.c.Hkv * a.c.page;
        if (d0 < a.c.dh) {   // dh % 32 == 0: a lane's dims lie in one block
            const float s = lp::pow2f(((const int8_t *)codes)[lines * a.c.dh + line * (a.c.dh / 32) + d0 / 32]);
            const uint8_t *src = codes + line * a.c.dh + d0;
            uint32_t w[(N + 3) / 4];
            if constexpr (N == 2) w[0] = *(const uint16_t *)src;
            else if constexpr (N == 4) w[0] = *(const uint32_t *)src;
            else if constexpr (N == 8) { const uint2 t = *(const uint2 *)src; w[0] = t.x; w[1] = t.y; }
            else { const uint4 t = *(const uint4 *)src; w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w; }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                __nv_fp8_e4m3 c;
                c.__x = (uint8_t)(w[i / 4] >> (8 * (i & 3)));
                f[i] = (float)c * s;
            }
        }
    } else {
        const S *src = (const S *)pages + line * a.c.dh + d0;
        constexpr int Q = N < 4 ? N : 4;   // dh is a multiple of 4: groups of four dims are all in or all out
#pragma unroll
        for (int i = 0; i < N; i += Q) {
            if (d0 + i < a.c.dh) {
                S e[Q];
                if constexpr (sizeof(S) * Q == 4) *reinterpret_cast<uint32_t *>(e) = *reinterpret_cast<const uint32_t *>(src + i);
                else if constexpr (sizeof(S) * Q == 8) *reinterpret_cast<uint2 *>(e) = *reinterpret_cast<const uint2 *>(src + i);
                else *reinterpret_cast<uint4 *>(e) = *reinterpret_cast<const uint4 *>(src + i);
#pragma unroll
                for (int q = 0; q < Q; ++q) f[i + q] = (float)e[q];
            }
        }
    }
}

template <typename S, bool FP8, int DH>
__global__ void __launch_bounds__(32 * kWarps) swa_decode_simt_kernel(DecodeArgs a, Split s) {
    constexpr int N = DH / 32, HB = heads_of<DH>(), NV = 4 * HB;
    extern __shared__ __align__(16) float sm_acc[];   // [kWarps][HB][DH]
    __shared__ float sm_m[kWarps][HB], sm_l[kWarps][HB];
    __shared__ int64_t sh[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = a.H / a.c.Hkv, blocks = (G + HB - 1) / HB;
    const float scale = a.scale * 1.4426950408889634f;

    Piece pc;
    if (s.direct) {
        pc.b = blockIdx.x / s.units_per_seq;
        pc.off = 0;
        pc.len = 1;
    } else {
        pc = piece_of<32 * kWarps, 16>(a, s, sh);
    }
    int64_t done = 0;
    while (done < pc.len) {
        const DecodeKeys<16> dk = decode_keys<16>(a.pos[pc.b], a.window, a.sinks, capacity_of(a), a.c.status);
        Segment sg;
        sg.b = pc.b;
        sg.n = dk.n;
        if (s.direct) {
            sg.u = blockIdx.x % s.units_per_seq;
            sg.c0 = 0;
            sg.c1 = dk.n;
            done = 1;
        } else {
            if (pc.off >= (int64_t)dk.n * s.units_per_seq) {   // next sequence (also past empty ones)
                pc.off = 0;
                ++pc.b;
                continue;
            }
            sg.u = (int)(pc.off / dk.n);
            sg.c0 = (int)(pc.off - (int64_t)sg.u * dk.n);
            const int64_t left = pc.len - done;
            sg.c1 = (int64_t)(dk.n - sg.c0) < left ? dk.n : sg.c0 + (int)left;
        }
        const int g = sg.u / blocks, h0 = (sg.u % blocks) * HB;
        const int heads = G - h0 < HB ? G - h0 : HB;
        // value lane: (key kg, head hd) of the halving exchange
        const int idx = lane / (32 / NV), hd = idx % HB, kg = idx / HB;
        float q[HB][N], acc[HB][N], m = -INFINITY, l = 0.f;
        const S *qr = (const S *)a.q + (int64_t)sg.b * a.ld_q + (int64_t)(g * G + h0) * a.c.dh;
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int d = lane * N + i;
                q[h][i] = h < heads && d < a.c.dh ? (float)qr[h * a.c.dh + d] * scale : 0.f;
                acc[h][i] = 0.f;
            }
        for (int c = sg.c0 + warp; c < sg.c1; c += kWarps) {
            const int j0 = dk.token(c);
            int id = a.c.table[(int64_t)sg.b * a.c.max_pages + j0 / a.c.page];
            if (id < 0 || id >= a.c.n_pages) {
                if (lane == 0) report(a.c.status, kStatusBounds);
                id = 0;
            }
            const int64_t line = ((int64_t)id * a.c.Hkv + g) * a.c.page + j0 % a.c.page;
            for (int t = 0; t < 16; t += 4) {
                bool any = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) any = any || dk.seen(j0 + t + i, a.sinks);
                if (!any) continue;
                float k[4][N], v[4][N];
#pragma unroll
                for (int i = 0; i < 4; ++i) load_row<S, FP8, DH>(a, a.c.k_pages, line + t + i, lane, k[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a row that is not seen is not read: it may hold anything
                    if (dk.seen(j0 + t + i, a.sinks)) load_row<S, FP8, DH>(a, a.c.v_pages, line + t + i, lane, v[i]);
                    else
#pragma unroll
                        for (int e = 0; e < N; ++e) v[i][e] = 0.f;
                }
                float r[NV];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        float x = 0.f;
#pragma unroll
                        for (int e = 0; e < N; ++e) x += q[h][e] * k[i][e];
                        r[i * HB + h] = x;
                    }
                int o = 16;
#pragma unroll
                for (int w = NV / 2; w; w >>= 1, o >>= 1) {
#pragma unroll
                    for (int i = 0; i < w; ++i) {
                        const bool up = lane & o;
                        const float keep = up ? r[i + w] : r[i], give = up ? r[i] : r[i + w];
                        r[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
                for (; o; o >>= 1) r[0] += __shfl_xor_sync(0xffffffffu, r[0], o);
                const float sc = dk.seen(j0 + t + kg, a.sinks) ? r[0] : -INFINITY;
                float mn = fmaxf(m, sc);   // of the head: its four lanes differ in the two upper bits
                mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 16));
                mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 8));
                const float ref = mn == -INFINITY ? 0.f : mn;
                const float f = m == -INFINITY ? 0.f : exp2f(m - ref);
                const float p = exp2f(sc - ref);
                const bool moved = __any_sync(0xffffffffu, mn != m);
                l = l * f + p;
                m = mn;
                if (moved) {
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        const float fh = __shfl_sync(0xffffffffu, f, h * (32 / NV));
#pragma unroll
                        for (int e = 0; e < N; ++e) acc[h][e] *= fh;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < HB; ++h) {
                        const float ph = __shfl_sync(0xffffffffu, p, (i * HB + h) * (32 / NV));
#pragma unroll
                        for (int e = 0; e < N; ++e) acc[h][e] += ph * v[i][e];
                    }
            }
        }
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        if (kg == 0 && lane % (32 / NV) == 0) {
            sm_m[warp][hd] = m;
            sm_l[warp][hd] = l;
        }
#pragma unroll
        for (int h = 0; h < HB; ++h)
#pragma unroll
            for (int e = 0; e < N; ++e) sm_acc[(warp * HB + h) * DH + lane * N + e] = acc[h][e];
        __syncthreads();
        const bool whole = sg.c1 - sg.c0 == sg.n;
        const int slot = done == 0 || s.direct ? 0 : 1;
        for (int i = threadIdx.x; i < heads * a.c.dh; i += 32 * kWarps) {
            const int h = i / a.c.dh, d = i - h * a.c.dh;
            float mm = -INFINITY, ll = 0.f, x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][h]);
            const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm_m[w][h] == -INFINITY ? 0.f : exp2f(sm_m[w][h] - ref);
                ll += sm_l[w][h] * f;
                x += sm_acc[(w * HB + h) * DH + d] * f;
            }
            if (whole) {
                S *dst = (S *)a.out + (int64_t)sg.b * a.ld_out + (int64_t)(g * G + h0 + h) * a.c.dh + d;
                store_val(dst, sg.n ? x / ll : 0.f);
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * HB + h;
                s.acc[at * a.c.dh + d] = x;
                if (d == 0) {
                    s.ml[2 * at] = mm;
                    s.ml[2 * at + 1] = ll;
                }
            }
        }
        __syncthreads();   // shared memory is written again by the next segment
        if (!s.direct) {
            done += sg.c1 - sg.c0;
            pc.off += sg.c1 - sg.c0;
        }
    }
}

// Joins the partials of one (unit, head) per block; empty slots get their zeros here.  Bound by the latency of its
// three dependent reads (prefix, (max, sum) pairs, O rows), so all of a read's loads are issued together: the
// pairs by all threads, then each warp takes every eighth row, kRows of them at a time.
constexpr int kJoinWarps = 8, kMaxParts = 2048;
template <typename S, int N>   // N: dims per lane (of dh <= 32 N)
__global__ void __launch_bounds__(32 * kJoinWarps) decode_join_kernel(DecodeArgs a, Split s, int HB, int grid) {
    constexpr int kRows = N <= 4 ? 8 : 2;
    const int G = a.H / a.c.Hkv, blocks = (G + HB - 1) / HB;
    const int b = blockIdx.x / a.H, hq = blockIdx.x % a.H, g = hq / G, hg = hq % G;
    const int u = g * blocks + hg / HB, h = hg % HB;
    const int64_t p0 = s.prefix[b], n = (s.prefix[b + 1] - p0) / s.units_per_seq, total = s.prefix[a.c.B];
    S *dst = (S *)a.out + (int64_t)b * a.ld_out + (int64_t)hq * a.c.dh;
    if (n == 0) {
        for (int d = threadIdx.x; d < a.c.dh; d += 32 * kJoinWarps) store_val(dst + d, 0.f);
        return;
    }
    const int64_t share = share_of(total, grid), t0 = p0 + u * n;
    const int first = (int)(t0 / share), last = (int)((t0 + n - 1) / share), parts = last - first + 1;
    if (parts == 1) return;   // finished by its CTA
    const bool late = t0 % share != 0;   // the unit starts inside its first CTA's piece: second slot
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto at = [&](int i) { return ((int64_t)(first + i) * 2 + (i == 0 && late ? 1 : 0)) * HB + h; };
    __shared__ float sm_f[kMaxParts], sm_m[kJoinWarps], sm_l[kJoinWarps];   // parts <= grid <= kMaxParts
    __shared__ float sm_x[kJoinWarps][32 * N];
    float m = -INFINITY;
    float2 ml[kMaxParts / (32 * kJoinWarps)];
#pragma unroll
    for (int i = 0; i < kMaxParts / (32 * kJoinWarps); ++i) {
        const int c = i * 32 * kJoinWarps + threadIdx.x;
        ml[i] = c < parts ? *reinterpret_cast<const float2 *>(s.ml + 2 * at(c)) : make_float2(-INFINITY, 0.f);
        m = fmaxf(m, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) sm_m[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sm_m[w]);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxParts / (32 * kJoinWarps); ++i) {
        const int c = i * 32 * kJoinWarps + threadIdx.x;
        if (c >= parts) break;
        const float f = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - ref);
        sm_f[c] = f;
        l += ml[i].y * f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane == 0) sm_l[warp] = l;
    __syncthreads();
    float x[N];
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
    for (int c0 = warp; c0 < parts; c0 += kJoinWarps * kRows) {
        float v[kRows][N];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int c = c0 + r * kJoinWarps;
#pragma unroll
            for (int e = 0; e < N; ++e)
                v[r][e] = c < parts && lane + 32 * e < a.c.dh ? s.acc[at(c) * a.c.dh + lane + 32 * e] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float f = c0 + r * kJoinWarps < parts ? sm_f[c0 + r * kJoinWarps] : 0.f;
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] += v[r][e] * f;
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sm_x[warp][lane + 32 * e] = x[e];
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += sm_l[w];
    for (int d = threadIdx.x; d < a.c.dh; d += 32 * kJoinWarps) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) y += sm_x[w][d];
        store_val(dst + d, y / l);
    }
}

template <typename S, bool FP8, int DH>
hcsa_status launch_simt(const DecodeArgs &a, cudaStream_t st) {
    constexpr int HB = heads_of<DH>(), smem = kWarps * HB * DH * (int)sizeof(float);
    static bool opted[64];
    if (!shared_opt_in((const void *)swa_decode_simt_kernel<S, FP8, DH>, smem, opted)) return HCSA_ERR_CUDA;
    const int G = a.H / a.c.Hkv, units = a.c.Hkv * ((G + HB - 1) / HB);
    const bool direct = decode_direct(a);
    if (direct && (int64_t)a.c.B * units > INT32_MAX) return HCSA_ERR_UNSUPPORTED;
    const int grid = direct ? a.c.B * units : sm_grid(kPerSM);
    Split s = make_split(a, units, HB, grid);
    s.direct = direct;
    swa_decode_simt_kernel<S, FP8, DH><<<grid, 32 * kWarps, smem, st>>>(a, s);
    count_launch();
    const hcsa_status r = check_launch();
    return r != HCSA_OK || direct ? r : launch_decode_join(a, s, HB, grid, st);
}

template <typename S, bool FP8>
hcsa_status launch_dh(const DecodeArgs &a, cudaStream_t st) {
    if (a.c.dh <= 64) return launch_simt<S, FP8, 64>(a, st);
    if (a.c.dh <= 128) return launch_simt<S, FP8, 128>(a, st);
    if (a.c.dh <= 256) return launch_simt<S, FP8, 256>(a, st);
    return launch_simt<S, FP8, 512>(a, st);
}

size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

}  // namespace

int decode_simt_heads(int dh) { return dh <= 256 ? 8 : 2; }

int sm_grid(int per_sm) {
    static int n[64] = {};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    if (!n[dev]) {
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) {
            cudaGetLastError();
            return per_sm * 148;
        }
        n[dev] = sms;
    }
    return per_sm * n[dev];
}

bool shared_opt_in(const void *kernel, int bytes, bool *done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64 && done[dev]) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return true;
}

size_t decode_split_bytes(int B, int grid, int heads, int dh) {
    return align256((size_t)(B + 1) * sizeof(int64_t)) + align256((size_t)grid * 2 * heads * 2 * sizeof(float)) +
           (size_t)grid * 2 * heads * dh * sizeof(float);
}

Split make_split(const DecodeArgs &a, int units_per_seq, int heads, int grid) {
    Split s{};
    s.units_per_seq = units_per_seq;
    uint8_t *w = (uint8_t *)a.ws;
    s.prefix = (int64_t *)w;
    w += align256((size_t)(a.c.B + 1) * sizeof(int64_t));
    s.ml = (float *)w;
    w += align256((size_t)grid * 2 * heads * 2 * sizeof(float));
    s.acc = (float *)w;
    return s;
}

// No unit reads more than kDirectTokens: the window's tokens and the first ones, in whole chunks of 16.
bool decode_direct(const DecodeArgs &a) {
    const int64_t cap = (int64_t)a.c.max_pages * a.c.page;
    const int64_t seen = ((int64_t)a.window + 30) / 16 * 16 + ((int64_t)a.sinks + 15) / 16 * 16;
    return (cap < seen ? cap : seen) <= kDirectTokens;
}

hcsa_status launch_decode_join(const DecodeArgs &a, const Split &s, int heads, int grid, cudaStream_t st) {
    if ((int64_t)a.c.B * a.H > INT32_MAX || grid > kMaxParts) return HCSA_ERR_UNSUPPORTED;
    const unsigned n = (unsigned)(a.c.B * a.H), t = 32 * kJoinWarps;
    auto run = [&](auto one) {
        using S = decltype(one);
        if (a.c.dh <= 64) decode_join_kernel<S, 2><<<n, t, 0, st>>>(a, s, heads, grid);
        else if (a.c.dh <= 128) decode_join_kernel<S, 4><<<n, t, 0, st>>>(a, s, heads, grid);
        else decode_join_kernel<S, 16><<<n, t, 0, st>>>(a, s, heads, grid);
    };
    if (a.c.dtype == HCSA_F32) run(float());
    else run(__nv_bfloat16());
    count_launch();
    return check_launch();
}

hcsa_status launch_decode_simt(const DecodeArgs &a, cudaStream_t st) {
    if (a.c.dtype == HCSA_F32) return launch_dh<float, false>(a, st);
    return a.c.lowprec ? launch_dh<__nv_bfloat16, true>(a, st) : launch_dh<__nv_bfloat16, false>(a, st);
}

size_t swa_decode_ws_bytes(int dtype, int B, int dh) {
    return decode_tc_supported(dtype, dh) ? decode_split_bytes(B, decode_tc_grid(), decode_tc_heads(), dh)
                                          : decode_split_bytes(B, sm_grid(kPerSM), decode_simt_heads(dh), dh);
}

hcsa_status launch_swa_decode(const DecodeArgs &a, cudaStream_t st) {
    return decode_tc_supported(a.c.dtype, a.c.dh) ? launch_decode_tc(a, st) : launch_decode_simt(a, st);
}

}  // namespace hcsa
