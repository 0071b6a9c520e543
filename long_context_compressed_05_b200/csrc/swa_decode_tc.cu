// One-token attention over the paged cache on the tensor cores: bf16 or FP8 pages, dh 64 or 128.
//
// One token per sequence gives each key row only H / Hkv uses, so the kernel is bound by reading the pages; the
// matrix instruction is the warp-wide m16n8k16 (16 query heads x 8 keys, then 16 heads x 8 channels), whose
// operands come from shared memory per warp: no CTA-wide step, no TMEM round trip, and 16 rows is what a group
// of heads fills, where tcgen05 would run 128 rows for them.
//
// Four warps take the chunks (16 tokens, or 32 of FP8 pages; never across a page) of a CTA's segment in turn.  Each warp runs its own
// ring of stages: lane 0 asks for a chunk's K and V by TMA boxes (hardware swizzle, so that ldmatrix reads without
// bank conflicts), 32 page ids are read at a time, and no warp waits for another until the segment's end, where
// the four (max, sum, O) are joined through the ring's memory.
//   S = Q K^T       Q fragments stay in registers for the segment
//   online softmax  a thread has 2 heads x 4 keys; O is rescaled only in chunks that raise a head's maximum
//   O += P V        S's accumulator layout is P's operand layout; P is rounded to bf16 (the sum is not)
// Keys that are not seen get weight 0, and their V rows are zeroed in shared memory before the product (0 x NaN is
// NaN); only chunks at the ends of the visible ranges have any.
//
// FP8 pages run the products in fp16, whose conversion from E4M3 is one instruction for two codes: a code times
// 2^(e - E), E a reference exponent of the warp, is an fp16 number when e lies in [E - 8, E + 7].  The K reference is
// picked again for a chunk that leaves the range; the V reference (O is held times 2^-E) is raised with O rescaled;
// a chunk whose exponents spread further takes the slow path: bf16 operands by full conversions.  Queries are scaled
// per head to fp16 by a power of two where that is exact (a ratio of 2^32 between the largest and the smallest
// channel), else the segment takes the slow path.  Weights are held times 2^11, so their rounding to fp16 is
// relative (2^-11) down to 2^-25 of the largest.  An infinite value is stored as 448 x 2^120 (drop_infinite): it is taken
// out of the product and its channel set at the end, since O is relative to the V reference and would come out finite.
// Codes 2i and 2i + 1 of a word share a register (K), or two keys'
// codes of one channel (V), so channels run in a permuted order that the Q fragments and the stores follow.
#include "decode_split.cuh"
#include "tc_common.cuh"

#include <cuda_fp16.h>

namespace hcsa {

namespace {

constexpr int kW = 4;                // warps
constexpr int kHB = 16;              // query heads of a unit
// CTAs per SM: the step's dependent latencies need about twelve warps.  That leaves 168 registers a thread, of which the
// FP8 kernel for dh 128 spills 12 to 24 bytes.
constexpr int kPerSM = 3;
constexpr int kRingBytes = 70 * 1024;

// CT: tokens per chunk.  FP8 chunks are 32 where the pages allow it: a step's instructions that do not grow with the
// chunk (waits, masks, maxima, page lines) were half of its issue slots at 16 (104 -> 86 us at 8 sequences up to 262144).
template <int DH, bool FP8, int CT> struct Shape {
    static constexpr int kTile = CT * DH * (FP8 ? 1 : 2);          // K or V of a chunk
    static constexpr int kStage = 2 * kTile;
    static constexpr int kStages = kRingBytes / (kW * kStage) < 8 ? kRingBytes / (kW * kStage) : 8;
    static constexpr int kExps = FP8 ? 2 * CT * (DH / 32) : 0;      // K's exponents, then V's
    static constexpr int kSmem = kW * kStages * (kStage + kExps) + 1024;
    static_assert(kStages >= 2 && kW * kHB * DH * 4 <= kW * kStages * kStage, "the join fits in the ring");
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

__device__ __forceinline__ void mma16816h(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2h(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// four codes -> two registers of two fp16 (codes 0, 1 and 2, 3), each times its factors
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t f01, uint32_t f23, uint32_t &r01, uint32_t &r23) {
    uint32_t x, y;
    asm("{.reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h;}"
        : "=r"(x), "=r"(y) : "r"(w));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r01) : "r"(x), "r"(f01));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r23) : "r"(y), "r"(f23));
}
// the same in bf16 for any exponent: scale factors s0 .. s3 of the codes
__device__ __forceinline__ void codes_bf16(uint32_t w, float s0, float s1, float s2, float s3, uint32_t &r01,
                                           uint32_t &r23) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_fp8_e4m3 c;
        c.__x = (uint8_t)(w >> (8 * i));
        v[i] = (float)c;
    }
    r01 = pack2(v[0] * s0, v[1] * s1);
    r23 = pack2(v[2] * s2, v[3] * s3);
}
__device__ __forceinline__ int max4s(uint32_t e) {   // largest of four signed bytes
    int m = (int8_t)e;
#pragma unroll
    for (int b = 1; b < 4; ++b) m = max(m, (int)(int8_t)(e >> (8 * b)));
    return m;
}
__device__ __forceinline__ float pow2_or_0(int e) { return e < -126 ? 0.f : lp::pow2f(e); }

// byte offset of granule g (16 bytes) of row r in a K or V tile, as the TMA box leaves it
template <int DH, bool FP8, int CT>
__device__ __forceinline__ uint32_t tile_offset(int r, int g) {
    if constexpr (FP8 && DH == 64) {          // 64-byte rows, 64-byte swizzle
        return r * 64 + ((g ^ ((r >> 1) & 3)) << 4);
    } else {                                  // 128-byte rows, 128-byte swizzle; bf16 dh 128: two such halves
        return (g >> 3) * (CT * 128) + tc::sw128_offset(r, g & 7);
    }
}

// FP8 values that no fp32 number holds (448 x 2^120 stands for infinity; NaN codes beside them) out of a chunk's V tile:
// their codes become zero, and cls, a bit per channel, takes their sign (positive ones first, then negative ones; NaN:
// both).  Every head gives every seen key a weight, so the class of a channel is the same for all.  Returns the row's
// exponents, the lowest one for a block without a code left, so that it does not raise the reference.  Out of line: it
// runs for chunks that hold an exponent of 120 or more.
template <int DH, int CT>
__device__ __noinline__ uint32_t drop_infinite(uint8_t *v, uint32_t exps, bool hidden, uint32_t *cls) {
    constexpr int NB = DH / 32;
    const int lane = threadIdx.x & 31, row = lane & (CT - 1);
    for (int b = 0; b < NB; ++b) {
        uint32_t pos = 0, neg = 0;
        const int e = (int8_t)(exps >> (8 * b));
        if (lane < CT && !hidden && e >= 120) {
            uint32_t left = 0;
            for (int w = 0; w < 8; ++w) {
                uint32_t *at = reinterpret_cast<uint32_t *>(v + tile_offset<DH, true, CT>(row, 2 * b + w / 4) + 4 * (w % 4));
                uint32_t codes = *at;
                for (int i = 0; i < 4; ++i) {
                    __nv_fp8_e4m3 c;
                    c.__x = (uint8_t)(codes >> (8 * i));
                    const float x = (float)c * lp::pow2f(e);
                    if (fabsf(x) < INFINITY) continue;
                    codes &= ~(0xFFu << (8 * i));
                    if (!(x < 0.f)) pos |= 1u << (4 * w + i);
                    if (!(x > 0.f)) neg |= 1u << (4 * w + i);
                }
                *at = codes;
                left |= codes & 0x7F7F7F7Fu;   // a negative value far below the scale is -0
            }
            if (!left) {
                for (int i = b; i < 4; i += NB)   // two blocks: their bytes come twice
                    exps = (exps & ~(0xFFu << (8 * i))) | (uint32_t)(uint8_t)-126 << (8 * i);
            }
        }
        pos = __reduce_or_sync(0xffffffffu, pos);
        neg = __reduce_or_sync(0xffffffffu, neg);
        if (lane == 0) {
            cls[b] |= pos;
            cls[NB + b] |= neg;
        }
    }
    tc::fence_async_smem();          // ordered before the next TMA write of this stage
    return __shfl_sync(0xffffffffu, exps, row);
}

template <int DH, bool FP8, int CT>
__global__ void __launch_bounds__(32 * kW, kPerSM)
swa_decode_tc_kernel(DecodeArgs a, Split s, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v) {
    using Sh = Shape<DH, FP8, CT>;
    constexpr int NST = Sh::kStages, NK = DH / 16, NB = DH / 32, NT = CT / 8;   // NT: score tiles of 8 keys
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t bars[kW][NST];
    __shared__ float sm_m[kW][kHB], sm_l[kW][kHB];
    __shared__ int64_t sh[kW];
    __shared__ uint32_t sm_cls[kW][2 * NB];   // FP8: channels with an infinite value (positive, negative)
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gr = lane >> 2, cq = lane & 3;
    const int G = a.H / a.c.Hkv, blocks = (G + kHB - 1) / kHB;
    const float scale = a.scale * 1.4426950408889634f;
    if (lane == 0) {
        for (int i = 0; i < NST; ++i) tc::mbar_init(&bars[warp][i], FP8 ? 33 : 1);   // FP8: every lane's exponent copies too
        tc::fence_mbar_init();
    }
    __syncwarp();
    const uint32_t stages = tc::smem_u32(ring) + warp * NST * Sh::kStage;
    uint8_t *exps = ring + kW * NST * Sh::kStage + warp * NST * Sh::kExps;
    const int64_t exps_at = (int64_t)a.c.n_pages * a.c.Hkv * a.c.page * DH;   // FP8: offset of the exponents
    uint32_t it = 0;                 // chunks this warp has asked for, over all segments
    uint32_t used = 0;               // chunks this warp has consumed
    bool ok = true;

    Piece pc;
    if (s.direct) {
        pc.b = blockIdx.x / s.units_per_seq;
        pc.off = 0;
        pc.len = 1;
    } else {
        pc = piece_of<32 * kW, CT>(a, s, sh);
    }
    int64_t done = 0;
    while (done < pc.len) {
        const DecodeKeys<CT> dk = decode_keys<CT>(a.pos[pc.b], a.window, a.sinks, capacity_of(a), a.c.status);
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
        if (FP8 && lane < 2 * NB) sm_cls[warp][lane] = 0;

        int lines = 0;               // lane i: first row of this warp's chunk (asked & ~31) + i in the page arrays
        int asked = 0;               // of this segment
        auto ask = [&]() {           // whole warp
            if ((asked & 31) == 0 && asked + lane < mine) {
                const int j0 = dk.token(sg.c0 + warp + (asked + lane) * kW), nth = j0 / a.c.page;
                int id = a.c.table[(int64_t)sg.b * a.c.max_pages + nth];
                if (id < 0 || id >= a.c.n_pages) {
                    report(a.c.status, kStatusBounds);
                    id = 0;
                }
                lines = (id * a.c.Hkv + g) * a.c.page + (j0 - nth * a.c.page);   // below 2^31 (checked on the host)
            }
            const int line = __shfl_sync(0xffffffffu, lines, asked & 31);
            if (lane == 0) {
                const int st = it % NST;
                const uint32_t dst = stages + st * Sh::kStage;
                uint64_t *bar = &bars[warp][st];
                tc::mbar_arrive_expect_tx(bar, Sh::kStage);
#pragma unroll
                for (int c = 0; c < (FP8 ? 1 : DH / 64); ++c) {
                    tc::tma_load_2d(dst + c * CT * 128, &tm_k, c * 64, line, bar);
                    tc::tma_load_2d(dst + Sh::kTile + c * CT * 128, &tm_v, c * 64, line, bar);
                }
            }
            if constexpr (FP8) {     // CT rows' exponents, contiguous: 16 bytes a lane, K's then V's
                constexpr int kVecs = Sh::kExps / 32;
                if (lane < 2 * kVecs) {
                    const uint8_t *src = (const uint8_t *)(lane < kVecs ? a.c.k_pages : a.c.v_pages) + exps_at +
                                         (int64_t)line * NB + (lane % kVecs) * 16;
                    tc::cp_async16(tc::smem_u32(exps + it % NST * Sh::kExps + lane * 16), src, true);
                }
                tc::cp_async_arrive_noinc(&bars[warp][it % NST]);
            }
            ++it;
            ++asked;
        };
        for (int i = 0; i < NST && i < mine; ++i) ask();

        // Q fragments: 16 heads x 16 channels a step; rows past the group are zero.  FP8: channels 4 cq .. + 3 of the
        // step, as its code words have them
        const __nv_bfloat16 *qr = (const __nv_bfloat16 *)a.q + (int64_t)sg.b * a.ld_q + (int64_t)(g * G + h0) * DH;
        auto load_q = [&](int k, uint32_t *f) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = gr + 8 * half;
                f[half] = f[2 + half] = 0;
                if (h >= heads) continue;
                if constexpr (FP8) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(qr + h * DH + 16 * k + 4 * cq));
                    f[half] = w.x;
                    f[2 + half] = w.y;
                } else {
                    f[half] = __ldg(reinterpret_cast<const uint32_t *>(qr + h * DH + 16 * k + 2 * cq));
                    f[2 + half] = __ldg(reinterpret_cast<const uint32_t *>(qr + h * DH + 16 * k + 8 + 2 * cq));
                }
            }
        };
        uint32_t q[NK][4];
#pragma unroll
        for (int k = 0; k < NK; ++k) load_q(k, q[k]);
        // FP8: to fp16 times 2^-up, the largest channel of a head in [2^14, 2^15)
        int up0 = 0, up1 = 0;
        bool q16 = false;
        if constexpr (FP8) {
            uint32_t big[2] = {0, 0};   // magnitude bits of bf16 order like the numbers
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    big[x & 1] = max(big[x & 1], max(q[k][x] & 0x7FFFu, (q[k][x] >> 16) & 0x7FFFu));
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                big[0] = max(big[0], __shfl_xor_sync(0xffffffffu, big[0], x));
                big[1] = max(big[1], __shfl_xor_sync(0xffffffffu, big[1], x));
            }
            q16 = big[0] < 0x7F80u && big[1] < 0x7F80u;   // finite
            up0 = q16 && big[0] ? (int)(big[0] >> 7) - 127 - 14 : 0;
            up1 = q16 && big[1] ? (int)(big[1] >> 7) - 127 - 14 : 0;
            q16 = q16 && abs(up0) < 64 && abs(up1) < 64;
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float f = lp::pow2f(q16 ? -(x & 1 ? up1 : up0) : 0);
                    const float lo = __uint_as_float(q[k][x] << 16) * f, hi = __uint_as_float(q[k][x] & 0xFFFF0000u) * f;
                    const uint32_t r = pack2h(lo, hi);
                    const __half2 back = *reinterpret_cast<const __half2 *>(&r);
                    q16 = q16 && __low2float(back) == lo && __high2float(back) == hi;
                    q[k][x] = r;
                }
            q16 = __all_sync(0xffffffffu, q16);
        }
        // weights are held times 2^kUp; with the maximum at most kSlack above the reference they stay below 2^15 (fp16)
        constexpr float kSlack = FP8 ? 4.f : 8.f, kUp = FP8 ? 11.f : 0.f, kUnUp = FP8 ? 0x1p-11f : 1.f;
        int Ek = 0, Ev = -128;       // reference exponents (Ev: none yet)
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
            const bool whole = dk.all_seen(j0, a.sinks);
            if (!whole) {            // V rows that are not seen: zeros
                for (int r = 0; r < CT; ++r) {
                    if (dk.seen(j0 + r, a.sinks)) continue;
                    uint8_t *v = ring + (warp * NST + st) * Sh::kStage + Sh::kTile;
                    if (lane < DH * (FP8 ? 1 : 2) / 16)
                        *reinterpret_cast<uint4 *>(v + tile_offset<DH, FP8, CT>(r, lane)) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_async_smem();   // ordered before the next TMA write of this stage
                __syncwarp();
            }
            // FP8: this lane's words of exponents against the references: z = 4 (e - E + 15) by byte, the upper byte of
            // the fp16 number 2^(e - E), where e - E is in [-8, 7]
            uint2 ew = make_uint2(0, 0);
            if constexpr (FP8) {     // K and V row lane % CT; unused bytes repeat used ones
                const uint8_t *ex = exps + st * Sh::kExps + (lane & (CT - 1)) * NB;
                if constexpr (NB == 4)
                    ew = make_uint2(*reinterpret_cast<const uint32_t *>(ex), *reinterpret_cast<const uint32_t *>(ex + CT * NB));
                else
                    ew = make_uint2(*reinterpret_cast<const uint16_t *>(ex) * 0x00010001u,
                                    *reinterpret_cast<const uint16_t *>(ex + CT * NB) * 0x00010001u);
            }
            uint2 z = ew;
            bool k_fast = q16, v_fast = true;
            if constexpr (FP8) {
                const bool hidden = !whole && !dk.seen(j0 + (lane & (CT - 1)), a.sinks);
                auto offset = [&](uint32_t e, int E, uint32_t &zz) {
                    const uint32_t d = hidden ? 0x08080808u : __vsub4(e, (uint32_t)((E - 8) & 255) * 0x01010101u);
                    zz = (d + 0x07070707u) << 2;
                    return !__any_sync(0xffffffffu, d & 0xF0F0F0F0u);
                };
                auto largest = [&](uint32_t e) { return __reduce_max_sync(0xffffffffu, hidden ? -126 : max4s(e)); };
                if (!offset(ew.x, Ek, z.x) && k_fast) {
                    const int top = largest(ew.x);
                    if (abs(top) < 60) Ek = top;
                    k_fast = offset(ew.x, Ek, z.x);
                }
                if (Ev == -128 || Ev > 112 || !offset(ew.y, Ev, z.y)) {   // an exponent of 120 comes here
                    if (__any_sync(0xffffffffu, !hidden && max4s(ew.y) >= 120)) {
                        __syncwarp();
                        ew.y = drop_infinite<DH, CT>(ring + (warp * NST + st) * Sh::kStage + Sh::kTile, ew.y, hidden, sm_cls[warp]);
                    }
                    const int top = largest(ew.y);
                    if (top > Ev) {
                        const float f = pow2_or_0(Ev - top);   // no value yet: O is zero
                        Ev = top;
#pragma unroll
                        for (int j = 0; j < 2 * NK; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[j][e] *= f;
                    }
                    v_fast = offset(ew.y, Ev, z.y);
                }
            }
            // word of tile t's key gr, and of keys 2 cq + (t & 1) + 8 (t / 2)
            auto k_word = [&](uint32_t w, int t) { return __shfl_sync(0xffffffffu, w, gr + 8 * t); };
            auto v_word = [&](uint32_t w, int t) { return __shfl_sync(0xffffffffu, w, 2 * cq + (t & 1) + 8 * (t >> 1)); };
            float sc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[t][e] = 0.f;
            if constexpr (!FP8) {
#pragma unroll
                for (int k = 0; k < NK; ++k)
#pragma unroll
                    for (int t = 0; t < NT; t += 2) {
                        uint32_t b[4];
                        ldsm4(kt + tile_offset<DH, FP8, CT>(8 * t + (lane & 7) + ((lane >> 4) & 1) * 8, 2 * k + ((lane >> 3) & 1)), b);
                        mma16816(sc[t], q[k], b[0], b[1]);
                        mma16816(sc[t + 1], q[k], b[2], b[3]);
                    }
            } else {
                uint32_t f[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t) f[t] = k_word(k_fast ? z.x : ew.x, t);
                if (k_fast) {
#pragma unroll
                    for (int k = 0; k < NK / 2; ++k)   // steps 2 k and 2 k + 1: block k
#pragma unroll
                        for (int t = 0; t < NT; t += 2) {
                            uint32_t w[4];
                            ldsm4(kt + tile_offset<DH, FP8, CT>(8 * t + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), w);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t b0, b1;
                                // byte k above a zero byte, twice
                                const uint32_t fk = __byte_perm(f[t + (e & 1)], 0, 0x0404 + 0x1010 * k);
                                codes_f16(w[e], fk, fk, b0, b1);
                                mma16816h(sc[t + (e & 1)], q[2 * k + (e >> 1)], b0, b1);
                            }
                        }
                } else {
                    for (int k = 0; k < NK / 2; ++k) {
                        uint32_t qb[2][4];
                        load_q(2 * k, qb[0]);
                        load_q(2 * k + 1, qb[1]);
#pragma unroll
                        for (int t = 0; t < NT; t += 2) {
                            uint32_t w[4];
                            ldsm4(kt + tile_offset<DH, FP8, CT>(8 * t + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * k + (lane >> 4)), w);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t b0, b1;
                                const float fk = lp::pow2f((int8_t)(f[t + (e & 1)] >> (8 * k)));
                                codes_bf16(w[e], fk, fk, fk, fk, b0, b1);
                                mma16816(sc[t + (e & 1)], qb[e >> 1], b0, b1);
                            }
                        }
                    }
                }
            }
            const bool scaled = FP8 && k_fast;   // undo the scales of Q and K
            const float s0 = scaled ? scale * lp::pow2f(up0 + Ek) : scale, s1 = scaled ? scale * lp::pow2f(up1 + Ek) : scale;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[t][e] *= e < 2 ? s0 : s1;
                    if (!whole && !dk.seen(j0 + 8 * t + 2 * cq + (e & 1), a.sinks)) sc[t][e] = -INFINITY;
                }
            float n0 = m0, n1 = m1;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                n0 = fmaxf(n0, fmaxf(sc[t][0], sc[t][1]));
                n1 = fmaxf(n1, fmaxf(sc[t][2], sc[t][3]));
            }
            // m is the reference of the exponentials, at most kSlack (exp2 units) below the maximum
            if (__any_sync(0xffffffffu, n0 > m0 + kSlack || n1 > m1 + kSlack)) {
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
                }
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
            const float r0 = m0 == -INFINITY ? 0.f : m0 - kUp, r1 = m1 == -INFINITY ? 0.f : m1 - kUp;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                sc[t][0] = ex2(sc[t][0] - r0);
                sc[t][1] = ex2(sc[t][1] - r0);
                sc[t][2] = ex2(sc[t][2] - r1);
                sc[t][3] = ex2(sc[t][3] - r1);
                l0 += sc[t][0] + sc[t][1];
                l1 += sc[t][2] + sc[t][3];
            }
            uint32_t p[CT / 16][4];
#pragma unroll
            for (int x = 0; x < CT / 16; ++x)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float lo = sc[2 * x + (t >> 1)][2 * (t & 1)], hi = sc[2 * x + (t >> 1)][2 * (t & 1) + 1];
                    p[x][t] = FP8 && v_fast ? pack2h(lo, hi) : pack2(lo, hi);
                }
            if constexpr (!FP8) {
#pragma unroll
                for (int x = 0; x < CT / 16; ++x)
#pragma unroll
                    for (int j = 0; j < NK; ++j) {
                        uint32_t b[4];
                        ldsm4t(vt + tile_offset<DH, FP8, CT>(16 * x + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * j + (lane >> 4)), b);
                        mma16816(o[2 * j], p[x], b[0], b[1]);
                        mma16816(o[2 * j + 1], p[x], b[2], b[3]);
                    }
            } else {
                // granules 2 j and 2 j + 1 of the row: block j.  A word of ldmatrix.trans: two channels of key 2 cq, then the
                // same of key 2 cq + 1 (t: keys 0..7, 8..15 of the 16)
#pragma unroll
                for (int x = 0; x < CT / 16; ++x) {
                    uint32_t fv[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) fv[t] = v_word(v_fast ? z.y : ew.y, 4 * x + t);
                    if (v_fast) {
#pragma unroll
                        for (int j = 0; j < NK / 2; ++j) {
                            uint32_t w[4], f[2];
                            ldsm4t(vt + tile_offset<DH, FP8, CT>(16 * x + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * j + (lane >> 4)), w);
#pragma unroll
                            for (int t = 0; t < 2; ++t)
                                f[t] = __byte_perm(fv[2 * t], fv[2 * t + 1], 0x4000 + 0x1010 * j) & 0xFF00FF00u;
#pragma unroll
                            for (int gi = 0; gi < 2; ++gi) {
                                uint32_t c0[2], c1[2];
#pragma unroll
                                for (int t = 0; t < 2; ++t)
                                    codes_f16(__byte_perm(w[2 * gi + t], 0, 0x3120), f[t], f[t], c0[t], c1[t]);
                                mma16816h(o[2 * (2 * j + gi)], p[x], c0[0], c0[1]);
                                mma16816h(o[2 * (2 * j + gi) + 1], p[x], c1[0], c1[1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < NK / 2; ++j) {
                            uint32_t w[4];
                            ldsm4t(vt + tile_offset<DH, FP8, CT>(16 * x + (lane & 7) + ((lane >> 3) & 1) * 8, 2 * j + (lane >> 4)), w);
#pragma unroll
                            for (int gi = 0; gi < 2; ++gi) {
                                uint32_t c0[2], c1[2];
#pragma unroll
                                for (int t = 0; t < 2; ++t) {
                                    // a row that is not seen has codes 0; its exponent may be anything
                                    const float fa = pow2_or_0(min((int8_t)(fv[2 * t] >> (8 * j)) - Ev, 127));
                                    const float fb = pow2_or_0(min((int8_t)(fv[2 * t + 1] >> (8 * j)) - Ev, 127));
                                    codes_bf16(__byte_perm(w[2 * gi + t], 0, 0x3120), fa, fb, fa, fb, c0[t], c1[t]);
                                }
                                mma16816(o[2 * (2 * j + gi)], p[x], c0[0], c0[1]);
                                mma16816(o[2 * (2 * j + gi) + 1], p[x], c1[0], c1[1]);
                            }
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
        if constexpr (FP8) {         // undo the weights' and V's references
            const float f = pow2_or_0(Ev);
            l0 *= kUnUp;
            l1 *= kUnUp;
#pragma unroll
            for (int j = 0; j < 2 * NK; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[j][e] = o[j][e] * kUnUp * f;
        }
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
        if constexpr (FP8) {
            __syncwarp();
            if (__any_sync(0xffffffffu, lane < 2 * NB && sm_cls[warp][lane % (2 * NB)]))
                for (int b = 0; b < NB; ++b) {
                    const bool pos = sm_cls[warp][b] >> lane & 1, neg = sm_cls[warp][NB + b] >> lane & 1;
                    for (int h = 0; (pos || neg) && h < kHB; ++h)   // added: a channel that is NaN already stays so
                        acc[(warp * kHB + h) * DH + 32 * b + lane] += pos && neg ? NAN : pos ? INFINITY : -INFINITY;
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

template <int DH, bool FP8, int CT>
hcsa_status launch(const DecodeArgs &a, cudaStream_t st) {
    using Sh = Shape<DH, FP8, CT>;
    auto kernel = swa_decode_tc_kernel<DH, FP8, CT>;
    static bool opted[64];
    if (!shared_opt_in((const void *)kernel, Sh::kSmem, opted)) return HCSA_ERR_CUDA;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)a.c.n_pages * a.c.Hkv * a.c.page;
    const bool made = FP8 ? make_tmap_u8_2d(&mk, a.c.k_pages, DH, rows, DH, DH, CT) &&
                                make_tmap_u8_2d(&mv, a.c.v_pages, DH, rows, DH, DH, CT)
                          : make_tmap_bf16_2d(&mk, a.c.k_pages, DH, rows, DH * 2, 64, CT, true) &&
                                make_tmap_bf16_2d(&mv, a.c.v_pages, DH, rows, DH * 2, 64, CT, true);
    if (!made) return HCSA_ERR_CUDA;
    const int G = a.H / a.c.Hkv, units = a.c.Hkv * ((G + kHB - 1) / kHB);
    const bool direct = decode_direct(a);
    if (direct && (int64_t)a.c.B * units > INT32_MAX) return HCSA_ERR_UNSUPPORTED;
    const int grid = direct ? a.c.B * units : sm_grid(kPerSM);
    Split s = make_split(a, units, kHB, grid);
    s.direct = direct;
    kernel<<<grid, 32 * kW, Sh::kSmem, st>>>(a, s, mk, mv);
    count_launch();
    const hcsa_status r = check_launch();
    return r != HCSA_OK || direct ? r : launch_decode_join(a, s, kHB, grid, st);
}

}  // namespace

int decode_tc_heads() { return kHB; }
int decode_tc_grid() { return sm_grid(kPerSM); }

// bf16 queries, dh 64 or 128 (any window, sinks, page and group)
bool decode_tc_supported(int dtype, int dh) { return dtype == HCSA_BF16 && (dh == 64 || dh == 128); }

hcsa_status launch_decode_tc(const DecodeArgs &a, cudaStream_t st) {
    if (!a.c.lowprec) return a.c.dh == 64 ? launch<64, false, 16>(a, st) : launch<128, false, 16>(a, st);
    if (a.c.page % 32 == 0) return a.c.dh == 64 ? launch<64, true, 32>(a, st) : launch<128, true, 32>(a, st);
    return a.c.dh == 64 ? launch<64, true, 16>(a, st) : launch<128, true, 16>(a, st);
}

}  // namespace hcsa
