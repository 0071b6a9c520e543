// One-token attention over the paged cache on the tensor cores: bf16 or FP8 pages, dh 64 or 128.
//
// One token per sequence gives each key row only H / Hkv uses, so the kernel is bound by reading the pages; the
// matrix instruction is the warp-wide m16n8k16 (16 query heads x 8 keys, then 16 heads x 8 channels), whose
// operands come from shared memory per warp: no CTA-wide step, no TMEM round trip, and 16 rows is what a group
// of heads fills, where tcgen05 would run 128 rows for them.
//
// Four warps take the chunks (16 tokens; never across a page) of a CTA's segment in turn.  Each warp runs its own
// ring of stages: lane 0 asks for a chunk's K and V by TMA boxes (hardware swizzle, so that ldmatrix reads without
// bank conflicts), 32 page ids are read at a time, and no warp waits for another until the segment's end, where
// the four (max, sum, O) are joined through the ring's memory.
//   S = Q K^T       Q fragments stay in registers for the segment
//   online softmax  a thread has 2 heads x 4 keys; O is rescaled only in chunks that raise a head's maximum
//   O += P V        S's accumulator layout is P's operand layout; P is rounded to bf16 (the sum is not)
// Keys that are not seen get weight 0, and their V rows are zeroed in shared memory before the product (0 x NaN is
// NaN); only chunks at the ends of the visible ranges have any.
//
// FP8 codes become bf16 operands exactly: the seven exponent and mantissa bits placed at the bottom of bf16's
// are the value times 2^-120, and one packed multiply by 2^(e + 120) restores it (blocks with e > 7 or NaN codes
// take the conversion instructions).  Codes 2i and 2i + 2 of a word share a register, so the K channels and the
// output channels run in a permuted order that the Q fragments and the stores follow.
#include "decode_split.cuh"
#include "tc_common.cuh"

namespace hcsa {

namespace {

constexpr int kW = 4;                // warps
constexpr int kHB = 16;              // query heads of a unit
constexpr int kRingBytes = 104 * 1024;   // two CTAs per SM

template <int DH, bool FP8> struct Shape {
    static constexpr int kTile = 16 * DH * (FP8 ? 1 : 2);          // K or V of a chunk
    static constexpr int kExps = FP8 ? 16 * (DH / 32) : 0;
    static constexpr int kStage = (2 * kTile + 2 * kExps + 1023) / 1024 * 1024;
    static constexpr int kStages = kRingBytes / (kW * kStage) < 8 ? kRingBytes / (kW * kStage) : 8;
    static constexpr int kTx = 2 * kTile + 2 * kExps;
    static constexpr int kSmem = kW * kStages * kStage + 1024;
    static_assert(kW * kHB * DH * 4 <= kW * kStages * kStage, "the join fits in the ring");
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four codes -> bf16 of codes (0, 2) and (1, 3), times the factors `f` (2^(e + 120), one per half)
__device__ __forceinline__ void codes_fast(uint32_t w, uint32_t f, uint32_t &even, uint32_t &odd) {
    even = mul2(((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u), f);
    odd = mul2(((w >> 4) & 0x07F007F0u) | (w & 0x80008000u), f);
}
// the same by conversion instructions, for any exponent and NaN codes: lo, hi the scales of the two halves
__device__ __forceinline__ void codes_any(uint32_t w, float lo, float hi, uint32_t &even, uint32_t &odd) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_fp8_e4m3 c;
        c.__x = (uint8_t)(w >> (8 * i));
        v[i] = (float)c * (i < 2 ? lo : hi);
    }
    // V: bytes 0, 1 are of the low halves' key, 2, 3 of the high halves'; K: one key, lo == hi
    even = pack2(v[0], v[2]);
    odd = pack2(v[1], v[3]);
}
// any code of the word that is NaN (0x7F or 0xFF) leaves a bit in the sign positions
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }
// any of four exponents above 7 (the factor 2^(e + 120) would pass bf16's range) leaves a bit in the sign positions
__device__ __forceinline__ uint32_t big_bits(uint32_t e) { return ((e & 0x78787878u) + 0x78787878u) & ~e; }
// e + 247 of four exponents up to 7: the exponent field of 2^(e + 120)
__device__ __forceinline__ uint32_t fields(uint32_t e) { return (e ^ 0x80808080u) + 0x77777777u; }

// byte offset of granule g (16 bytes) of row r in a K or V tile, as the TMA box leaves it
template <int DH, bool FP8>
__device__ __forceinline__ uint32_t tile_offset(int r, int g) {
    if constexpr (FP8 && DH == 64) {          // 64-byte rows, 64-byte swizzle
        return r * 64 + ((g ^ ((r >> 1) & 3)) << 4);
    } else {                                  // 128-byte rows, 128-byte swizzle; bf16 dh 128: two such halves
        return (g >> 3) * 2048 + tc::sw128_offset(r, g & 7);
    }
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(32 * kW, 2)
swa_decode_tc_kernel(DecodeArgs a, Split s, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
    using Sh = Shape<DH, FP8>;
    constexpr int NST = Sh::kStages, NK = DH / 16, NB = DH / 32;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kW][NST];
    __shared__ float sm_m[kW][kHB], sm_l[kW][kHB];
    __shared__ int64_t sh[kW];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gr = lane >> 2, cq = lane & 3;
    const int G = a.H / a.c.Hkv, blocks = (G + kHB - 1) / kHB;
    const float scale = a.scale * 1.4426950408889634f;
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) tc::mbar_init(&bars[warp][i], 1);
        tc::fence_mbar_init();
    }
    __syncwarp();
    const uint32_t stages = tc::smem_u32(ring) + warp * NST * Sh::kStage;
    uint32_t it = 0;                 // chunks this warp has asked for, over all segments
    uint32_t used = 0;               // chunks this warp has consumed
    bool ok = true;

    Piece pc;
    if (s.direct) {
        pc.b = blockIdx.x / s.units_per_seq;
        pc.off = 0;
        pc.len = 1;
    } else {
        pc = piece_of<32 * kW>(a, s, sh);
    }
    int64_t done = 0;
    while (done < pc.len) {
        const DecodeKeys dk = decode_keys(a.pos[pc.b], a.window, a.sinks, capacity_of(a), a.c.status);
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
        const int g = sg.u / blocks, h0 = (sg.u % blocks) * kHB;
        const int heads = G - h0 < kHB ? G - h0 : kHB;
        const int mine = sg.c1 - sg.c0 > warp ? (sg.c1 - sg.c0 - warp + kW - 1) / kW : 0;   // chunks of this warp

        int ids = 0;                 // lane i: page of this warp's chunk (asked & ~31) + i
        int asked = 0;               // of this segment
        auto ask = [&]() {           // whole warp
            if ((asked & 31) == 0) {
                ids = 0;
                if (asked + lane < mine) {
                    const int j0 = dk.token(sg.c0 + warp + (asked + lane) * kW);
                    ids = a.c.table[(int64_t)sg.b * a.c.max_pages + j0 / a.c.page];
                    if (ids < 0 || ids >= a.c.n_pages) {
                        report(a.c.status, kStatusBounds);
                        ids = 0;
                    }
                }
            }
            const int id = __shfl_sync(0xffffffffu, ids, asked & 31);
            if (lane == 0) {
                const int j0 = dk.token(sg.c0 + warp + asked * kW);
                const int line = (id * a.c.Hkv + g) * a.c.page + j0 % a.c.page;   // below 2^31 (checked on the host)
                const int st = it % NST;
                const uint32_t dst = stages + st * Sh::kStage;
                uint64_t *bar = &bars[warp][st];
                tc::mbar_arrive_expect_tx(bar, Sh::kTx);
#pragma unroll
                for (int c = 0; c < (FP8 ? 1 : DH / 64); ++c) {
                    tc::tma_load_2d(dst + c * 2048, &tm_k, c * 64, line, bar);
                    tc::tma_load_2d(dst + Sh::kTile + c * 2048, &tm_v, c * 64, line, bar);
                }
                if constexpr (FP8) {
                    const int64_t lines = (int64_t)a.c.n_pages * a.c.Hkv * a.c.page;
                    const int64_t at = lines * DH + (int64_t)line * NB;
                    tc::bulk_load(dst + 2 * Sh::kTile, (const uint8_t *)a.c.k_pages + at, Sh::kExps, bar);
                    tc::bulk_load(dst + 2 * Sh::kTile + Sh::kExps, (const uint8_t *)a.c.v_pages + at, Sh::kExps, bar);
                }
            }
            ++it;
            ++asked;
        };
        for (int i = 0; i < NST && i < mine; ++i) ask();

        // Q fragments: 16 heads x 16 channels a step; rows past the group are zero
        uint32_t q[NK][4];
        {
            const __nv_bfloat16 *qr = (const __nv_bfloat16 *)a.q + (int64_t)sg.b * a.ld_q + (int64_t)(g * G + h0) * DH;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = gr + 8 * half;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    if constexpr (FP8) {   // channels 4 cq .. + 3 of the step: (0, 2) then (1, 3)
                        uint2 w = make_uint2(0, 0);
                        if (h < heads) w = __ldg(reinterpret_cast<const uint2 *>(qr + h * DH + 16 * k + 4 * cq));
                        q[k][half] = __byte_perm(w.x, w.y, 0x5410);
                        q[k][2 + half] = __byte_perm(w.x, w.y, 0x7632);
                    } else {
                        q[k][half] = q[k][2 + half] = 0;
                        if (h < heads) {
                            q[k][half] = __ldg(reinterpret_cast<const uint32_t *>(qr + h * DH + 16 * k + 2 * cq));
                            q[k][2 + half] = __ldg(reinterpret_cast<const uint32_t *>(qr + h * DH + 16 * k + 8 + 2 * cq));
                        }
                    }
                }
            }
        }
        float o[2 * NK][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;   // heads gr and gr + 8
#pragma unroll
        for (int i = 0; i < 2 * NK; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

        for (int i = 0; i < mine && ok; ++i, ++used) {
            const int st = used % NST;
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[warp][st], (used / NST) & 1, a.c.status));
            if (!ok) break;
            const uint32_t kt = stages + st * Sh::kStage, vt = kt + Sh::kTile;
            const int j0 = dk.token(sg.c0 + warp + i * kW);
            const bool whole = token_seen(dk, j0, a.sinks) && token_seen(dk, j0 + 15, a.sinks) &&
                               (j0 >= dk.w0 || j0 + 15 < a.sinks);
            // the exponents of the four keys and two key columns this thread touches
            uint32_t ke[2] = {0, 0}, ve[4] = {0, 0, 0, 0};
            if constexpr (FP8) {
                const uint8_t *ex = ring + (warp * NST + st) * Sh::kStage + 2 * Sh::kTile;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if constexpr (NB == 4) ke[t] = *reinterpret_cast<const uint32_t *>(ex + (gr + 8 * t) * 4);
                    else ke[t] = *reinterpret_cast<const uint16_t *>(ex + (gr + 8 * t) * 2);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = 2 * cq + e + 8 * t;
                        if constexpr (NB == 4) ve[2 * t + e] = *reinterpret_cast<const uint32_t *>(ex + Sh::kExps + row * 4);
                        else ve[2 * t + e] = *reinterpret_cast<const uint16_t *>(ex + Sh::kExps + row * 2);
                    }
                }
            }
            if (!whole) {            // rows that are not seen: V to zero (FP8: codes and exponents)
                for (int r = 0; r < 16; ++r) {
                    if (token_seen(dk, j0 + r, a.sinks)) continue;
                    uint8_t *v = ring + (warp * NST + st) * Sh::kStage + Sh::kTile;
                    if (lane < Sh::kTile / 256)
                        *reinterpret_cast<uint4 *>(v + tile_offset<DH, FP8>(r, lane)) = make_uint4(0, 0, 0, 0);
                    if constexpr (FP8) {
                        // exponents of K and V: the products of the zeros and of masked keys must not take the slow path
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (gr + 8 * t == r) ke[t] = 0;
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (2 * cq + e + 8 * t == r) ve[2 * t + e] = 0;
                        }
                    }
                }
                tc::fence_async_smem();   // ordered before the next TMA write of this stage
                __syncwarp();
            }
            float sc[2][4], sd[2][4];   // even and odd steps: two shorter chains of products
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[t][e] = sd[t][e] = 0.f;
            if constexpr (!FP8) {
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    uint32_t b[4];
                    ldsm4(kt + tile_offset<DH, FP8>((lane & 7) + ((lane >> 4) & 1) * 8, 2 * k + ((lane >> 3) & 1)), b);
                    mma16816(k & 1 ? sd[0] : sc[0], q[k], b[0], b[1]);
                    mma16816(k & 1 ? sd[1] : sc[1], q[k], b[2], b[3]);
                }
            } else {
                uint32_t w[NK / 2][4], nan = 0;
#pragma unroll
                for (int k = 0; k < NK / 2; ++k) {
                    ldsm4(kt + tile_offset<DH, FP8>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), w[k]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) nan |= nan_bits(w[k][e]);
                }
                if (!__any_sync(0xffffffffu, (nan | big_bits(ke[0]) | big_bits(ke[1])) & 0x80808080u)) {
                    const uint32_t z[2] = {fields(ke[0]), fields(ke[1])};
#pragma unroll
                    for (int k = 0; k < NK / 2; ++k) {   // steps 2 k and 2 k + 1: block k
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b0, b1;
                            // byte k of z in both halves, in the place of a bf16 exponent
                            codes_fast(w[k][e], __byte_perm(z[e & 1], 0, 0x4040 + 0x0101 * k) << 7, b0, b1);
                            mma16816(e >> 1 ? sd[e & 1] : sc[e & 1], q[2 * k + (e >> 1)], b0, b1);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < NK / 2; ++k) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b0, b1;
                            const float f = lp::pow2f((int8_t)(ke[e & 1] >> (8 * k)));
                            codes_any(w[k][e], f, f, b0, b1);
                            mma16816(e >> 1 ? sd[e & 1] : sc[e & 1], q[2 * k + (e >> 1)], b0, b1);
                        }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[t][e] = (sc[t][e] + sd[t][e]) * scale;
                    if (!whole && !token_seen(dk, j0 + 8 * t + 2 * cq + (e & 1), a.sinks)) sc[t][e] = -INFINITY;
                }
            float n0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
            float n1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
            }
            n0 = fmaxf(n0, m0);
            n1 = fmaxf(n1, m1);
            if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {
                // -inf - -inf: a head without a finite score yet has no sum to rescale
                const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int j = 0; j < 2 * NK; ++j) {
                    o[j][0] *= f0;
                    o[j][1] *= f0;
                    o[j][2] *= f1;
                    o[j][3] *= f1;
                }
            }
            const float r0 = m0 == -INFINITY ? 0.f : m0, r1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sc[t][0] = ex2(sc[t][0] - r0);
                sc[t][1] = ex2(sc[t][1] - r0);
                sc[t][2] = ex2(sc[t][2] - r1);
                sc[t][3] = ex2(sc[t][3] - r1);
                l0 += sc[t][0] + sc[t][1];
                l1 += sc[t][2] + sc[t][3];
            }
            const uint32_t p[4] = {pack2(sc[0][0], sc[0][1]), pack2(sc[0][2], sc[0][3]), pack2(sc[1][0], sc[1][1]),
                                   pack2(sc[1][2], sc[1][3])};
            if constexpr (!FP8) {
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    uint32_t b[4];
                    ldsm4t(vt + tile_offset<DH, FP8>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * j + (lane >> 4)), b);
                    mma16816(o[2 * j], p, b[0], b[1]);
                    mma16816(o[2 * j + 1], p, b[2], b[3]);
                }
            } else {
                uint32_t w[NK / 2][4], nan = 0;
#pragma unroll
                for (int j = 0; j < NK / 2; ++j) {
                    ldsm4t(vt + tile_offset<DH, FP8>((lane & 7) + ((lane >> 3) & 1) * 8, 2 * j + (lane >> 4)), w[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) nan |= nan_bits(w[j][e]);
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) nan |= big_bits(ve[t]);
                // granules 2 j and 2 j + 1 of the row: block j; t: keys 0..7, 8..15
                if (!__any_sync(0xffffffffu, nan & 0x80808080u)) {
                    const uint32_t z[4] = {fields(ve[0]), fields(ve[1]), fields(ve[2]), fields(ve[3])};
#pragma unroll
                    for (int j = 0; j < NK / 2; ++j) {
                        uint32_t f[2];
#pragma unroll
                        for (int t = 0; t < 2; ++t) f[t] = (__byte_perm(z[2 * t], z[2 * t + 1], 0x0400 + 0x0101 * j) & 0x00FF00FFu) << 7;
#pragma unroll
                        for (int gi = 0; gi < 2; ++gi) {
                            uint32_t e0[2], o0[2];
#pragma unroll
                            for (int t = 0; t < 2; ++t) codes_fast(w[j][2 * gi + t], f[t], e0[t], o0[t]);
                            mma16816(o[2 * (2 * j + gi)], p, e0[0], e0[1]);
                            mma16816(o[2 * (2 * j + gi) + 1], p, o0[0], o0[1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < NK / 2; ++j) {
#pragma unroll
                        for (int gi = 0; gi < 2; ++gi) {
                            uint32_t e0[2], o0[2];
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                codes_any(w[j][2 * gi + t], lp::pow2f((int8_t)(ve[2 * t] >> (8 * j))),
                                          lp::pow2f((int8_t)(ve[2 * t + 1] >> (8 * j))), e0[t], o0[t]);
                            mma16816(o[2 * (2 * j + gi)], p, e0[0], e0[1]);
                            mma16816(o[2 * (2 * j + gi) + 1], p, o0[0], o0[1]);
                        }
                    }
                }
            }
            __syncwarp();            // every lane has read the stage
            if (asked < mine) ask();
        }

        // ------------------------------------------------ join of the warps
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        if (cq == 0) {
            sm_m[warp][gr] = m0;
            sm_m[warp][gr + 8] = m1;
            sm_l[warp][gr] = l0;
            sm_l[warp][gr + 8] = l1;
        }
        ok = __syncthreads_and(ok);  // no copy in flight and every warp is done with the ring (or all give up)
        if (!ok) break;
        float *acc = reinterpret_cast<float *>(ring);   // [kW][kHB][DH]
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float *dst = acc + (warp * kHB + gr + 8 * half) * DH;
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                if constexpr (FP8) {   // even and odd channels of the step's 16
                    *reinterpret_cast<float4 *>(dst + 16 * j + 4 * cq) =
                        make_float4(o[2 * j][2 * half], o[2 * j + 1][2 * half], o[2 * j][2 * half + 1],
                                    o[2 * j + 1][2 * half + 1]);
                } else {
                    *reinterpret_cast<float2 *>(dst + 16 * j + 2 * cq) =
                        make_float2(o[2 * j][2 * half], o[2 * j][2 * half + 1]);
                    *reinterpret_cast<float2 *>(dst + 16 * j + 8 + 2 * cq) =
                        make_float2(o[2 * j + 1][2 * half], o[2 * j + 1][2 * half + 1]);
                }
            }
        }
        __syncthreads();
        const bool whole_unit = sg.c1 - sg.c0 == sg.n;
        const int slot = done == 0 || s.direct ? 0 : 1;
        for (int i = threadIdx.x * 2; i < heads * DH; i += 64 * kW) {
            const int h = i / DH, d = i - h * DH;
            float mm = -INFINITY, ll = 0.f;
            float2 x = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kW; ++w) mm = fmaxf(mm, sm_m[w][h]);
            const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const float f = sm_m[w][h] == -INFINITY ? 0.f : ex2(sm_m[w][h] - ref);
                const float2 v = *reinterpret_cast<const float2 *>(acc + (w * kHB + h) * DH + d);
                ll += sm_l[w][h] * f;
                x.x += v.x * f;
                x.y += v.y * f;
            }
            if (whole_unit) {
                __nv_bfloat16 *dst =
                    (__nv_bfloat16 *)a.out + (int64_t)sg.b * a.ld_out + (int64_t)(g * G + h0 + h) * DH + d;
                *reinterpret_cast<uint32_t *>(dst) = sg.n ? pack2(x.x / ll, x.y / ll) : 0u;
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * kHB + h;
                *reinterpret_cast<float2 *>(s.acc + at * DH + d) = x;
                if (d == 0) {
                    s.ml[2 * at] = mm;
                    s.ml[2 * at + 1] = ll;
                }
            }
        }
        tc::fence_async_smem();      // these accesses of the ring come before the next segment's TMA writes
        __syncthreads();
        if (!s.direct) {
            done += sg.c1 - sg.c0;
            pc.off += sg.c1 - sg.c0;
        }
    }
    // given up: wait (bounded) for the copies still in flight before the shared memory goes away
    for (; used < it; ++used)
        tc::mbar_wait(&bars[warp][used % NST], (used / NST) & 1, a.c.status);
}

template <int DH, bool FP8>
hcsa_status launch(const DecodeArgs &a, cudaStream_t st) {
    using Sh = Shape<DH, FP8>;
    auto kernel = swa_decode_tc_kernel<DH, FP8>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess)
        return HCSA_ERR_CUDA;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)a.c.n_pages * a.c.Hkv * a.c.page;
    const bool made = FP8 ? make_tmap_u8_2d(&mk, a.c.k_pages, DH, rows, DH, DH, 16) &&
                                make_tmap_u8_2d(&mv, a.c.v_pages, DH, rows, DH, DH, 16)
                          : make_tmap_bf16_2d(&mk, a.c.k_pages, DH, rows, DH * 2, 64, 16, true) &&
                                make_tmap_bf16_2d(&mv, a.c.v_pages, DH, rows, DH * 2, 64, 16, true);
    if (!made) return HCSA_ERR_CUDA;
    const int G = a.H / a.c.Hkv, units = a.c.Hkv * ((G + kHB - 1) / kHB);
    const bool direct = decode_direct(a);
    if (direct && (int64_t)a.c.B * units > INT32_MAX) return HCSA_ERR_UNSUPPORTED;
    const int grid = direct ? a.c.B * units : decode_grid();
    Split s = make_split(a, units, kHB, grid);
    s.direct = direct;
    kernel<<<grid, 32 * kW, Sh::kSmem, st>>>(a, s, mk, mv);
    count_launch();
    const hcsa_status r = check_launch();
    return r != HCSA_OK || direct ? r : launch_decode_join(a, s, kHB, grid, st);
}

}  // namespace

int decode_tc_heads() { return kHB; }

// bf16 queries, dh 64 or 128 (any window, sinks, page and group)
bool decode_tc_supported(int dtype, int dh) { return dtype == HCSA_BF16 && (dh == 64 || dh == 128); }

hcsa_status launch_decode_tc(const DecodeArgs &a, cudaStream_t st) {
    if (a.c.dh == 64) return a.c.lowprec ? launch<64, true>(a, st) : launch<64, false>(a, st);
    return a.c.lowprec ? launch<128, true>(a, st) : launch<128, false>(a, st);
}

}  // namespace hcsa
