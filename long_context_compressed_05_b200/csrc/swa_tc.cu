// Sliding-window prefill attention on the tensor cores (tcgen05 + TMEM, TMA box loads): bf16, dh 64 or 128, any group of
// heads, window and first tokens.
//
// A block is two sub-tiles of 128 query rows of one key head: a row is a (token, head of the group) pair, a sub-tile
// holds floor(128 / G) tokens.  Both sub-tiles walk the same tiles of 128 key columns (the first tokens outside the
// window, padded to 16, then the tokens from the first row's window on; see block_keys) and share their loads.
//   S = Q K^T        128 x 128 fp32 in TMEM, one buffer per sub-tile
//   online softmax   a warpgroup per sub-tile, a thread per row (no exchange between threads); the running maximum is
//                    raised, and O rescaled in TMEM, only when a row's maximum grows by more than 2^8
//   O += P V         P (bf16) as the A operand in TMEM, written over S and handed over in two parts (96 + 32 columns), so
//                    that only the last 32 keys' products are left when the softmax ends; V an MN-major B operand
// Each sub-tile has its own issuing warp.  They take turns, and a turn issues the end of a P V and the next S behind it
// (also across blocks), so that one sub-tile's products run while the other's softmax does.  Persistent CTAs take the
// blocks longest first, in a snake order over the CTAs.  Warps: 0 and 3 TMA, 1 and 2 MMA, 4..7 and 8..11 softmax and
// output of sub-tile 0 and 1.
//
// Per tile of 128 x 128 at dh 128 the products take 1024 cycles of the tensor core and the exponentials 1024 of the
// special-function unit: two equal bounds for a long window.  What holds it above them is the chain of a sub-tile (S,
// softmax, P V, next S), of which TMEM has room for two.  Measured at 8192 tokens, 32 heads over 8, dh 128, causal: 406 to
// 418 us (1340 TFLOP/s), captured.  What was tried there, beside 409: P in one part 462; parts of 64 + 64 462, four of 32
// 479; two threads per row 466; two S buffers of 64 columns 458 (the narrow products are bound by shared memory); a
// quarter of the exponentials by a polynomial on the FMA pipe 441; one issuing warp for both sub-tiles 497.  A window of
// 128 (65536 tokens, 64 heads over 8, dh 128: 690 us) is bound by the same chain: two tiles a block, then the output.
// These are at 1965 MHz; seconds of such calls run at the power limit, 1500 to 1660 MHz (480 and 820 us).  dh 64, 8192
// tokens, 32 heads over 8, causal: 349 us (788 TFLOP/s), by the exponentials: half the products for as many of them.
#include "sliding.cuh"
#include "tc_common.cuh"

namespace hcsa {

namespace {

constexpr int kRows = 128;           // query rows of a sub-tile
constexpr int kKT = 128;             // key columns of a tile
constexpr int kGran = 16;            // rows of the small TMA boxes: padding of the first tokens' columns
constexpr int kGroups = 4;           // groups of 32 key columns
constexpr int kEarly = 3;            // of them, those whose P is handed over before the last one's is ready
constexpr int kThreads = 384;
// Registers a thread: 168 at launch (384 threads), shared out anew as 80 for the TMA / MMA warpgroup and 208 for
// the two softmax warpgroups (128 x 80 + 256 x 208 <= 384 x 168)
constexpr int kRegsIssue = 80, kRegsSoftmax = 208;
constexpr uint32_t kColO = 256;      // TMEM: S (later P) of sub-tile s at 128 s, O at 256 + 128 s
constexpr float kSlack = 8.f;        // exp2 units

struct Args {
    SwaArgs a;
    int G, tb;                       // heads per key head, tokens per sub-tile
    bool wide;                       // output rows start on 32-byte boundaries
    uint32_t blocks, n_units;        // blocks of tokens, x key heads
    float scale_log2;
};

template <int DH> struct Sizes {
    static constexpr int kChunk = kRows * 128;              // 128 rows x 64 bf16
    static constexpr int kTile = DH / 64 * kChunk;          // Q, K or V tile
    static constexpr int kStages = DH == 128 ? 2 : 4;       // of K and of V
    static constexpr int kSmem = 2 * kTile + 2 * kStages * kTile + 2048;
};

template <int NST> struct Bars {
    uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST];
    uint64_t q_full[2], q_empty[2], s_full[2], p_early[2], p_full[2], o_full[2], o_empty[2], turn[2], drain[2];
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// An issuing warp runs its loop with all lanes and no branch around the products, so that addresses and descriptors
// stay in uniform registers: a product takes about 30 cycles to issue, against 60 in a branch of one lane and 120
// where one lane runs the whole loop.  `leader` is 1 in the elected lane.
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
    return r;
}
// D[tmem] (+)= A[smem] B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc),
                 "r"(accumulate), "r"(leader)
                 : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A's row i in lane i, two bf16 per 32-bit column
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t at, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(at), "l"(bdesc), "r"(idesc),
                 "r"(accumulate), "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
                 "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void expect(uint32_t leader, uint64_t *bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %2, 0;\n\t"
                 "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(tc::smem_u32(bar)), "r"(bytes),
                 "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void load_2d(uint32_t leader, uint32_t dst, const CUtensorMap *map, int c0, int c1, uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                 "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
                 "[%4];\n\t}" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(tc::smem_u32(bar)),
                 "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t leader, uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                        uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %6, 0;\n\t"
                 "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
                 "%4}], [%5];\n\t}" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2),
                 "r"(tc::smem_u32(bar)), "r"(leader)
                 : "memory");
}
__device__ __forceinline__ void arrive(uint32_t leader, uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t@e mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(
                     tc::smem_u32(bar)), "r"(leader)
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float &x, float &y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void store32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// Key columns of a block, the same in every role.
struct Cols {
    int pad, sk;                     // the window part starts at column pad; columns below sk are first tokens
    int n_tiles;
    int hi0, hi1, lo0, lo1;          // of each sub-tile: its last column (-1: no tokens), its first window column
    __device__ __forceinline__ int hi(int s) const { return s ? hi1 : hi0; }
    // does sub-tile s see a column of tile i?
    __device__ __forceinline__ bool active(int s, int i) const {
        const int c0 = i * kKT;
        return c0 <= hi(s) && (c0 < sk || c0 + kKT - 1 >= (s ? lo1 : lo0));
    }
};
struct Unit {
    int g, t0, t_end, w0;            // key head, tokens, first token of the window part
    Cols c;
    __device__ __forceinline__ int first(int s, int tb) const { return t0 + s * tb; }
    __device__ __forceinline__ int last(int s, int tb) const { return min(t0 + (s + 1) * tb, t_end) - 1; }
    // window columns of token t
    __device__ __forceinline__ int hi(int t) const { return t - w0 + c.pad; }
    __device__ __forceinline__ int lo(int t, int window) const { return t - window + 1 - w0 + c.pad; }
};

__device__ __forceinline__ Unit unit_of(const Args &p, uint32_t u) {
    const SwaArgs &a = p.a;
    Unit x;
    const uint32_t block = u / (uint32_t)a.Hkv;
    x.g = (int)(u - block * a.Hkv);
    x.t0 = a.row0 + (int)(p.blocks - 1 - block) * 2 * p.tb;   // longest first
    x.t_end = min(x.t0 + 2 * p.tb, a.row1);
    const BlockKeys b = block_keys(x.t0, x.t_end - 1, a.window, a.sinks, kGran);
    // the first tokens may reach the window: one run of columns from token 0
    const bool run = b.pad >= b.w0;
    x.w0 = run ? 0 : b.w0;
    x.c.pad = run ? 0 : b.pad;
    x.c.sk = run ? a.sinks : b.n_sink;
    x.c.n_tiles = (x.hi(x.t_end - 1) + kKT) / kKT;
    x.c.hi0 = x.hi(x.last(0, p.tb));
    x.c.hi1 = x.first(1, p.tb) < x.t_end ? x.hi(x.last(1, p.tb)) : -1;
    x.c.lo0 = x.lo(x.t0, a.window);
    x.c.lo1 = x.lo(x.first(1, p.tb), a.window);
    return x;
}
// k-th block of this CTA, or -1
__device__ __forceinline__ int nth_unit(const Args &p, int k) {
    const uint32_t u = (uint32_t)k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    return u < p.n_units ? (int)u : -1;
}

__device__ __forceinline__ void mma16816(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// bits 15 and 31: which of a word's two bf16 is infinite or NaN (its exponent all ones: the sum carries)
__device__ __forceinline__ uint32_t bad_halves(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// 16 rows from row r0 of sub-tile s, those in `rows`, once more over the keys that they see, by one warp.  Infinite and
// NaN values leave the product (as zeros) and reach the rows that see them at the end: an infinite channel if all that a
// row sees there have one sign, else NaN.  Operands straight from global memory, 16 keys at a time; lane (gr, cq) of
// a product reads dims cq DH/4 .. of its rows and keys, and channels gr DH/8 .. of its values, so that its words are
// contiguous, and holds channels cq DH/4 .. of output rows gr and gr + 8.
template <int DH>
__device__ __forceinline__ void attend_rows(const Args &p, const Unit &x, int s, int r0, uint32_t rows, int lane) {
    constexpr int NK = DH / 16, NJ = DH / 8, NO = DH / 4;   // steps over dims, products over channels, channels of a lane
    constexpr uint32_t kAll = NO == 32 ? ~0u : (1u << (NO & 31)) - 1u;
    using bf16 = __nv_bfloat16;
    const SwaArgs &a = p.a;
    const int gr = lane >> 2, cq = lane & 3;
    const int t_min = x.first(s, p.tb) + (r0 + __ffs(rows) - 1) / p.G, t_max = x.first(s, p.tb) + (r0 + 31 - __clz(rows)) / p.G;
    const int w_lo = t_min - a.window + 1 > 0 ? t_min - a.window + 1 : 0, far = a.sinks < w_lo ? a.sinks : w_lo;
    const int n = far + (t_max - w_lo + 1);
    auto token = [&](int c) -> int64_t { return c < far ? c : w_lo + (c - far); };
    int t[2];                        // -1: not a row to compute
    int64_t at[2];                   // head of the row, in q and out columns
    uint32_t q[NK][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + gr + 8 * i;
        t[i] = rows >> (gr + 8 * i) & 1 ? x.first(s, p.tb) + r / p.G : -1;
        at[i] = (int64_t)(x.g * p.G + r % p.G) * DH;
        const bf16 *src = (const bf16 *)a.q + (t[i] < 0 ? 0 : t[i] * a.ld_q + at[i]) + cq * NO;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const uint2 w = t[i] < 0 ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2 *>(src + 4 * k));
            q[k][i] = w.x;
            q[k][2 + i] = w.y;
        }
    }
    auto seen = [&](int i, int c) {
        const int64_t j = token(c);
        return c < n && j <= t[i] && (j > (int64_t)t[i] - a.window || j < a.sinks);
    };
    const bf16 *kb = (const bf16 *)a.k + x.g * DH + cq * NO, *vb = (const bf16 *)a.v + x.g * DH;
    float o[NJ][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    uint32_t pos[2] = {0, 0}, neg[2] = {0, 0};   // a bit per channel of the lane: infinite values seen, by sign (NaN: both)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
    for (int c0 = 0; c0 < n; c0 += 16) {
        auto row_of = [&](int c) { return token(c < n ? c : n - 1); };   // columns past the end weigh nothing
        float sc[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[h][e] = 0.f;
            const bf16 *src = kb + row_of(c0 + 8 * h + gr) * a.ld_k;
#pragma unroll
            for (int k = 0; k < NK; k += 2) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src + 4 * k));
                mma16816(sc[h], q[k], w.x, w.y);
                mma16816(sc[h], q[k + 1], w.z, w.w);
            }
        }
        uint32_t v[4][NJ / 2];       // keys 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9
        uint32_t any = 0;
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const bf16 *src = vb + row_of(c0 + 2 * cq + (y & 1) + 8 * (y >> 1)) * a.ld_v + gr * NJ;
#pragma unroll
            for (int w = 0; w < NJ / 2; w += 4) {
                const uint4 r = __ldg(reinterpret_cast<const uint4 *>(src + 2 * w));
                v[y][w] = r.x;
                v[y][w + 1] = r.y;
                v[y][w + 2] = r.z;
                v[y][w + 3] = r.w;
            }
#pragma unroll
            for (int w = 0; w < NJ / 2; ++w) {
                const uint32_t bad = bad_halves(v[y][w]);
                v[y][w] &= ~((bad >> 15) * 0xFFFFu);
                any |= bad;
            }
        }
        if (__any_sync(0xffffffffu, any)) {
            for (int c = c0; c < c0 + 16 && c < n; ++c) {
                const bf16 *src = vb + token(c) * a.ld_v + cq * NO;
                uint32_t up = 0, down = 0;
#pragma unroll
                for (int i = 0; i < NO; i += 8) {
                    const uint4 r = __ldg(reinterpret_cast<const uint4 *>(src + i));
                    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
                        const uint32_t bit = fabsf(f) < INFINITY ? 0u : 1u << (i + e);
                        if (!(f < 0.f)) up |= bit;
                        if (!(f > 0.f)) down |= bit;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (seen(i, c)) {
                        pos[i] |= up;
                        neg[i] |= down;
                    }
            }
            // every row NaN in every channel: no further key changes that
            if (__all_sync(0xffffffffu, (t[0] < 0 || (pos[0] & neg[0]) == kAll) && (t[1] < 0 || (pos[1] & neg[1]) == kAll))) break;
        }
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc[h][e] = seen(e >> 1, c0 + 8 * h + 2 * cq + (e & 1)) ? sc[h][e] * p.scale_log2 : -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], sc[h][e]);
            }
        float f[2], ref[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            f[i] = m[i] == -INFINITY ? 0.f : ex2(m[i] - mx[i]);
            ref[i] = mx[i] == -INFINITY ? 0.f : mx[i];
            m[i] = mx[i];
            l[i] *= f[i];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc[h][e] = ex2(sc[h][e] - ref[e >> 1]);
                l[e >> 1] += sc[h][e];
            }
        const uint32_t pw[4] = {pack2(sc[0][0], sc[0][1]), pack2(sc[0][2], sc[0][3]), pack2(sc[1][0], sc[1][1]),
                                pack2(sc[1][2], sc[1][3])};
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] *= f[e >> 1];
            const uint32_t half = j & 1 ? 0x7632 : 0x5410;
            mma16816(o[j], pw, __byte_perm(v[0][j / 2], v[1][j / 2], half), __byte_perm(v[2][j / 2], v[3][j / 2], half));
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        const float li = 1.f / l[i];
        // channel c of the lane: product c % NJ, column c / NJ of its pair
        auto value = [&](int c) {
            const float y = o[c % NJ][2 * i + c / NJ] * li;
            const bool up = pos[i] >> c & 1, down = neg[i] >> c & 1;
            return !(up || down) || !(l[i] > 0.f) ? y : up && down ? NAN : up ? INFINITY : -INFINITY;
        };
        if (t[i] < 0) continue;
        bf16 *dst = (bf16 *)a.out + t[i] * a.ld_out + at[i] + cq * NO;
#pragma unroll
        for (int c = 0; c < NO; c += 8)
            *reinterpret_cast<uint4 *>(dst + c) = make_uint4(pack2(value(c), value(c + 1)), pack2(value(c + 2), value(c + 3)),
                                                             pack2(value(c + 4), value(c + 5)), pack2(value(c + 6), value(c + 7)));
    }
}

template <int DH>
__device__ __forceinline__ __nv_bfloat16 *out_row(const Args &p, const Unit &x, int s, int row) {
    const int tl = row / p.G;
    return (__nv_bfloat16 *)p.a.out + (x.first(s, p.tb) + tl) * p.a.ld_out + (int64_t)(x.g * p.G + row - tl * p.G) * DH;
}
// Rows (of the 32 from r0 of sub-tile s, those in `rows`, tokens ta .. te) of which a channel is finite, so that their weights
// are, and whose other channels each have an infinite or NaN value that the row sees: the class of those values is all that
// there is to set, and a pass over the values finds it.  Returns the rows set.
template <int DH>
__device__ __forceinline__ uint32_t class_rows(const Args &p, const Unit &x, int s, int r0, uint32_t rows, int ta, int te, int lane) {
    constexpr int NW = DH / 64;      // words of a lane: channels 2 NW lane ..
    const SwaArgs &a = p.a;
    struct Class {                   // a bit per half-word (15 and 31): infinite values by sign, NaN both
        uint32_t up[NW], down[NW];
    };
    auto see = [&](int64_t j, Class &c) {
        const uint32_t *v = reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)a.v + j * a.ld_v + x.g * DH) + NW * lane;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const uint32_t r = __ldg(v + w), b = bad_halves(r);
            if (!b) continue;
            const uint32_t nan = (((r & 0x007F007Fu) + 0x007F007Fu) & 0x00800080u) << 8 & b;   // a mantissa bit
            c.up[w] |= (b & ~r) | nan;
            c.down[w] |= (b & r) | nan;
        }
    };
    Class core{};                    // of the tokens that all of ta .. te see
#pragma unroll 8
    for (int j = 0; j < a.sinks && j <= ta && j <= te - a.window; ++j) see(j, core);
#pragma unroll 8
    for (int j = te - a.window + 1 > 0 ? te - a.window + 1 : 0; j <= ta; ++j) see(j, core);
    uint32_t done = 0;
    for (uint32_t left = rows; left; left &= left - 1) {
        const int i = __ffs(left) - 1, t = x.first(s, p.tb) + (r0 + i) / p.G;
        Class c = core;
        for (int j = t - a.window + 1 > 0 ? t - a.window + 1 : 0; j <= ta && j <= te - a.window; ++j) see(j, c);
        for (int j = ta + 1; j <= t; ++j)
            if (j > t - a.window || j < a.sinks) see(j, c);
        uint32_t *o = reinterpret_cast<uint32_t *>(out_row<DH>(p, x, s, r0 + i)) + NW * lane;
        uint32_t bad[NW];
        bool open = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            bad[w] = bad_halves(o[w]);
            open = open || (bad[w] & ~(c.up[w] | c.down[w]));
        }
        if (__any_sync(0xffffffffu, open)) continue;
        done |= 1u << i;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const uint32_t both = c.up[w] & c.down[w] & bad[w], all = (bad[w] >> 15) * 0xFFFFu;
            // infinity 7F80, with its sign; NaN: a mantissa bit more
            if (bad[w]) o[w] = (o[w] & ~all) | (all & 0x7F807F80u) | (bad[w] & c.down[w] & ~both) | both >> 9;
        }
    }
    return done;
}

// Is a value of key head g in tokens [lo, hi) infinite or NaN?
template <int DH>
__device__ bool values_bad(const SwaArgs &a, int g, int64_t lo, int64_t hi, int lane) {
    uint32_t bad = 0;
    for (int64_t j = lo; j < hi; ++j)
        for (int d = 2 * lane; d < DH; d += 64)
            bad |= bad_halves(__ldg(reinterpret_cast<const uint32_t *>((const __nv_bfloat16 *)a.v + j * a.ld_v + g * DH + d)));
    return __any_sync(0xffffffffu, bad);
}

// The products give every masked key the weight 0, and 0 times an infinite or NaN value is NaN.  So the rows of sub-tile s,
// lanes [32 quad, 32 quad + 32), of this CTA's blocks that came out non-finite are computed again where a value that their
// block loaded and not all of them see is infinite or NaN.  By the warp that has stored them, once it has handed over its
// last block: nothing waits for it any more.  (Rows take as long as they have keys, the pipeline's waits are bounded.)
template <int DH>
__device__ __noinline__ void redo_rows(const Args &p, int s, int quad, int lane) {
    const SwaArgs &a = p.a;
    for (int k = 0;; ++k) {
        const int u = nth_unit(p, k);
        if (u < 0) break;
        const Unit x = unit_of(p, u);
        const int row = 32 * quad + lane, tl = row / p.G;
        uint32_t b = 0, all = 0x80008000u;
        if (tl < p.tb && x.first(s, p.tb) + tl <= x.last(s, p.tb)) {
            const uint4 *o = reinterpret_cast<const uint4 *>(out_row<DH>(p, x, s, row));
#pragma unroll
            for (int d = 0; d < DH / 8; ++d) {
                const uint4 r = o[d];
                const uint32_t h[4] = {bad_halves(r.x), bad_halves(r.y), bad_halves(r.z), bad_halves(r.w)};
                b |= h[0] | h[1] | h[2] | h[3];
                all &= h[0] & h[1] & h[2] & h[3];
            }
        }
        uint32_t bad = __ballot_sync(0xffffffffu, b);
        const uint32_t some = __ballot_sync(0xffffffffu, all != 0x80008000u);   // a channel is finite (of either half)
        if (!bad) continue;
        const int ta = x.first(s, p.tb) + (32 * quad + __ffs(bad) - 1) / p.G, te = x.first(s, p.tb) + (32 * quad + 31 - __clz(bad)) / p.G;
        const int behind = min(a.row1, x.w0 + x.c.n_tiles * kKT - x.c.pad);   // tokens loaded for the block
        if (!values_bad<DH>(a, x.g, x.w0, (int64_t)te - a.window + 1, lane) && !values_bad<DH>(a, x.g, ta + 1, behind, lane) &&
            !(x.c.pad && values_bad<DH>(a, x.g, x.c.sk, x.c.pad, lane)))
            continue;
        if (bad & some) bad &= ~class_rows<DH>(p, x, s, 32 * quad, bad & some, ta, te, lane);
        for (int half = 0; half < 2; ++half)
            if (bad >> (16 * half) & 0xFFFFu) attend_rows<DH>(p, x, s, 32 * quad + 16 * half, bad >> (16 * half) & 0xFFFFu, lane);
    }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
swa_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
              const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ Args p) {
    using Sz = Sizes<DH>;
    constexpr int NST = Sz::kStages, NC = DH / 64;
    constexpr uint32_t kIdescS = tc::idesc_bf16(128, kKT, false, false);
    constexpr uint32_t kIdescPV = tc::idesc_bf16(128, DH, false, true);
    const SwaArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    Bars<NST> *bars = reinterpret_cast<Bars<NST> *>(smem_raw);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 1);
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tmem_slot + 4) + 1023) & ~uintptr_t(1023));
    const uint32_t Qs = tc::smem_u32(base), Ks = Qs + 2 * Sz::kTile, Vs = Ks + NST * Sz::kTile;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            tc::mbar_init(&bars->k_full[i], 1);
            tc::mbar_init(&bars->k_empty[i], 2);   // both issuers
            tc::mbar_init(&bars->v_full[i], 1);
            tc::mbar_init(&bars->v_empty[i], 2);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&bars->q_full[s], 1);
            tc::mbar_init(&bars->q_empty[s], 1);
            tc::mbar_init(&bars->s_full[s], 1);
            tc::mbar_init(&bars->p_early[s], 4);
            tc::mbar_init(&bars->p_full[s], 4);
            tc::mbar_init(&bars->o_full[s], 1);
            tc::mbar_init(&bars->o_empty[s], 4);
            tc::mbar_init(&bars->turn[s], 1);
            tc::mbar_init(&bars->drain[s], 1);
        }
        tc::fence_mbar_init();
    }
    if (warp == 0) tc::tmem_alloc(tmem_slot, 512);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);   // uniform
    bool ok = true;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        const uint32_t leader = elect();
        auto wait = [&](uint64_t *bar, uint32_t parity) { ok = ok && tc::mbar_wait(bar, parity, a.status); };
        if (warp == 0 || warp == 3) {
            // ------------------------------------------------------ TMA: Q and K (warp 0), V (warp 3)
            const bool is_v = warp == 3;
            const CUtensorMap *map = is_v ? &tm_v : &tm_k, *map16 = is_v ? &tm_v16 : &tm_k16;
            uint64_t *full = is_v ? bars->v_full : bars->k_full, *empty = is_v ? bars->v_empty : bars->k_empty;
            const uint32_t ring = is_v ? Vs : Ks;
            uint32_t it = 0, n = 0, nq0 = 0, nq1 = 0;   // tiles; loads issued
            auto load_q = [&](const Unit &x, int s, uint32_t &nq) {
                if (is_v || x.c.hi(s) < 0) return;
                if (nq) wait(&bars->q_empty[s], (nq - 1) & 1);
                if (!ok) return;
                expect(leader, &bars->q_full[s], NC * 128 * p.tb * p.G);
                for (int c = 0; c < NC; ++c)
                    load_3d(leader, Qs + s * Sz::kTile + c * Sz::kChunk, &tm_q, c * 64, x.g * p.G, x.first(s, p.tb),
                            &bars->q_full[s]);
                ++nq;
            };
            for (int k = 0; ok; ++k) {
                const int u = nth_unit(p, k);
                if (u < 0) break;
                const Unit x = unit_of(p, u);
                load_q(x, 0, nq0);
                for (int i = 0; i < x.c.n_tiles && ok; ++i, ++it) {
                    const int st = it % NST, c0 = i * kKT;
                    if (it >= NST) wait(&empty[st], (it / NST - 1) & 1);
                    if (!ok) break;
                    const uint32_t dst = ring + st * Sz::kTile;
                    expect(leader, &full[st], Sz::kTile);
                    for (int c = 0; c < NC; ++c) {
                        const int x0 = x.g * DH + c * 64;
                        if (c0 >= x.c.pad) {
                            load_2d(leader, dst + c * Sz::kChunk, map, x0, x.w0 + c0 - x.c.pad, &full[st]);
                        } else {
                            for (int r = 0; r < kKT; r += kGran)
                                load_2d(leader, dst + c * Sz::kChunk + r * 128, map16, x0,
                                        c0 + r < x.c.pad ? c0 + r : x.w0 + c0 + r - x.c.pad, &full[st]);
                        }
                    }
                    ++n;
                    if (i == 0) load_q(x, 1, nq1);
                }
            }
            // given up: the copies still in flight land (bounded waits) before the shared memory goes away
            if (!ok) {
                for (uint32_t j = n > NST ? n - NST : 0; j < n; ++j)
                    tc::mbar_wait(&full[j % NST], (j / NST) & 1, a.status);
                if (nq0) tc::mbar_wait(&bars->q_full[0], (nq0 - 1) & 1, a.status);
                if (nq1) tc::mbar_wait(&bars->q_full[1], (nq1 - 1) & 1, a.status);
            }
        } else {
            // ------------------------------------------------------ MMA issuer of sub-tile s
            const int s = warp - 1;
            const uint64_t qd = tc::sdesc_sw128(Qs + s * Sz::kTile, 16, 1024), k0 = tc::sdesc_sw128(Ks, 16, 1024),
                           v0 = tc::sdesc_sw128(Vs, Sz::kChunk, 1024);
            const uint32_t tS = tmem + s * 128, tO = tmem + kColO + s * 128;
            uint32_t it = 0, np = 0, nu = 0, nt = 0;   // tiles, P tiles of the sub-tile, blocks that have it, turns taken
            // The P V that the sub-tile's last tile still owes
            bool owed = false, act = false, first = false, last = false;
            uint32_t vst = 0, vpar = 0;
            auto issue_pv = [&](int from, int to, uint64_t *bar) {   // groups of keys
                const uint64_t vd = v0 + vst * (Sz::kTile >> 4);
                wait(bar, np & 1);
                if (!ok) return;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 2 * from; k < 2 * to; ++k)
                    mma_ts(leader, tO, tS + 8 * k, vd + 128 * k, kIdescPV, !first || k != 0 ? 1u : 0u);
            };
            auto before_turn = [&]() {
                if (!owed) return;
                wait(&bars->v_full[vst], vpar);
                if (!act) return;
                if (first && nu > 1) wait(&bars->o_empty[s], nu & 1);   // of the block before this one
                issue_pv(0, kEarly, &bars->p_early[s]);
            };
            auto take_turn = [&]() {
                if (s == 1 || nt) wait(&bars->turn[s], (s == 1 ? nt : nt - 1) & 1);
                ++nt;
                if (!ok) return;
                if (owed && act) {
                    issue_pv(kEarly, kGroups, &bars->p_full[s]);
                    if (last) commit(leader, &bars->o_full[s]);
                    ++np;
                }
                tc::tc_fence_after();
            };
            for (int kk = 0; ok; ++kk) {
                const int u = nth_unit(p, kk);
                if (u < 0) break;
                const Cols c = unit_of(p, u).c;
                const int end = c.hi(s) < 0 ? -1 : c.hi(s) / kKT;   // its last tile is always active
                bool fresh = true;
                for (int i = 0; i < c.n_tiles; ++i, ++it) {
                    const int st = it % NST;
                    const bool now = c.active(s, i);
                    const uint64_t kd = k0 + st * (Sz::kTile >> 4);
                    // waited for also where the sub-tile does not use the tile: the stage's next use is told apart by it
                    wait(&bars->k_full[st], (it / NST) & 1);
                    if (now && fresh) wait(&bars->q_full[s], nu & 1);
                    before_turn();
                    take_turn();
                    if (!ok) break;
                    if (now) {
#pragma unroll
                        for (int k = 0; k < DH / 16; ++k) {
                            constexpr int kC = Sz::kChunk >> 4;
                            mma_ss(leader, tS, qd + (k >> 2) * kC + 2 * (k & 3), kd + (k >> 2) * kC + 2 * (k & 3), kIdescS,
                                   k != 0 ? 1u : 0u);
                        }
                        commit(leader, &bars->s_full[s]);
                    }
                    arrive(leader, &bars->turn[s ^ 1]);
                    if (now && i == end) commit(leader, &bars->q_empty[s]);
                    if (owed) commit(leader, &bars->v_empty[vst]);
                    commit(leader, &bars->k_empty[st]);
                    owed = true;
                    act = now;
                    first = fresh;
                    last = i == end;
                    vst = st;
                    vpar = (it / NST) & 1;
                    if (now) {
                        if (fresh) ++nu;
                        fresh = false;
                    }
                }
            }
            if (ok) {
                before_turn();
                if (ok) take_turn();
                arrive(leader, &bars->turn[s ^ 1]);
            }
            if (!ok) {               // given up: the products in flight end (bounded wait) before their memory goes away
                commit(leader, &bars->drain[s]);
                tc::mbar_wait(&bars->drain[s], 0, a.status);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------------------------------------------------- softmax + output: a thread per row
        const int s = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), tS = lanes + s * 128, tO = lanes + kColO + s * 128;
        const int tl = r / p.G, hh = r - tl * p.G;
        uint32_t ns = 0, nu = 0;     // steps and blocks seen
        bool bad = false;            // an output of this thread's rows is not finite
        for (int kk = 0; ok; ++kk) {
            const int u = nth_unit(p, kk);
            if (u < 0) break;
            const Unit x = unit_of(p, u);
            if (x.c.hi(s) < 0) continue;
            const int ta = x.first(s, p.tb), te = x.last(s, p.tb), t = ta + tl;
            const bool row_ok = tl < p.tb && t <= te;
            const int hi = row_ok ? x.hi(t) : -1, lo = row_ok ? x.lo(t, a.window) : 0;
            float m = -INFINITY, l = 0.f;
            bool first = true;
            // tiles between these columns are seen whole by every row
            const int clean_hi = x.hi(ta) - kKT + 1, clean_lo = x.lo(te, a.window), end = x.c.hi(s) / kKT;
            for (int i = 0; i <= end; ++i) {
                if (!x.c.active(s, i)) continue;
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars->s_full[s], ns & 1, a.status));
                if (!ok) break;
                tc::tc_fence_after();
                float v[kKT];
#pragma unroll
                for (int c = 0; c < kKT; c += 32) tc::tmem_ld32(tS + c, v + c);
                tc::tmem_ld_wait();
                // columns c0 + 32 q + c that the row sees, bit c; groups of 32 that no row of the warp sees are left out, and
                // weigh nothing
                const int c0 = i * kKT;
                const bool clean = c0 <= clean_hi && (c0 >= clean_lo || c0 + kKT <= x.c.sk);
                unsigned groups = 15;
                if (!clean) {
                    auto upto = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        const int cg = c0 + 32 * q;
                        const uint32_t bits = upto(hi + 1 - cg) & (~upto(lo - cg) | upto(x.c.sk - cg));
                        if (!__any_sync(0xffffffffu, bits)) {
                            groups &= ~(1u << q);
                        } else if (!__all_sync(0xffffffffu, bits == ~0u)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(bits >> c & 1)) v[32 * q + c] = -INFINITY;
                        }
                    }
                }
                auto group_max = [&](int q) {
                    float mx[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx[e] = fmaxf(v[32 * q + e], v[32 * q + e + 4]);
#pragma unroll
                    for (int c = 8; c < 32; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], v[32 * q + c + e], v[32 * q + c + e + 4]);
                    return max3(mx[0], mx[1], fmaxf(mx[2], mx[3]));
                };
                float mt = -INFINITY;
                if (groups == 15) {
                    mt = max3(group_max(0), group_max(1), fmaxf(group_max(2), group_max(3)));
                } else {
#pragma unroll
                    for (int q = 0; q < kGroups; ++q)
                        if (groups >> q & 1) mt = fmaxf(mt, group_max(q));
                }
                mt *= p.scale_log2;
                const bool need = mt > m + kSlack;
                if (__any_sync(0xffffffffu, need)) {
                    const float m_new = need ? mt : m;
                    if (!first) {    // s_full also says that the previous P V has completed
                        const float f = need ? ex2(m - m_new) : 1.f;   // m = -inf: 0
                        l *= f;
                        float o[32];
#pragma unroll
                        for (int c = 0; c < DH; c += 32) {
                            tc::tmem_ld32(tO + c, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f;
                            tc::tmem_st32(tO + c, o);
                        }
                    }
                    m = m_new;
                }
                first = false;
                ++ns;
                const float ref = m == -INFINITY ? 0.f : m;   // a row that has seen no key yet: every weight 0
                const uint64_t sc2 = f2(p.scale_log2, p.scale_log2), ref2 = f2(-ref, -ref);
                uint64_t sum[4] = {0, 0, 0, 0};   // pairs of zeros
                auto weigh = [&](int q, float *w) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float e0, e1;
                        unf2(fma2(f2(v[32 * q + 2 * c], v[32 * q + 2 * c + 1]), sc2, ref2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum[c & 3] = add2(sum[c & 3], f2(e0, e1));
                        w[c] = __uint_as_float(pack2(e0, e1));
                    }
                };
                auto hand_over = [&](uint64_t *bar) {
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(bar);
                };
                float w[16];
                if (groups == 15) {  // without branches between the groups
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        weigh(q, w);
                        tc::tmem_st16(tS + 16 * q, w);
                        if (q == kEarly - 1) hand_over(&bars->p_early[s]);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < kGroups; ++q) {
                        if (groups >> q & 1) {
                            weigh(q, w);
                        } else {
#pragma unroll
                            for (int c = 0; c < 16; ++c) w[c] = 0.f;
                        }
                        tc::tmem_st16(tS + 16 * q, w);
                        if (q == kEarly - 1) hand_over(&bars->p_early[s]);
                    }
                }
                hand_over(&bars->p_full[s]);
                float s0, s1;
                unf2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
                l += s0 + s1;
            }
            if (!ok) break;
            // ------------------------------------------------ output
            ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars->o_full[s], nu & 1, a.status));
            if (!ok) break;
            ++nu;
            tc::tc_fence_after();
            __nv_bfloat16 *dst = (__nv_bfloat16 *)a.out + (int64_t)t * a.ld_out + (int64_t)(x.g * p.G + hh) * DH;
            const float li = 1.f / l;
            uint64_t zero = 0;       // NaN once an output is not finite
#pragma unroll
            for (int c = 0; c < DH; c += 64) {
                float o[64];
                tc::tmem_ld32(tO + c, o);
                tc::tmem_ld32(tO + c + 32, o + 32);
                tc::tmem_ld_wait();
                if (c + 64 == DH) {  // O is read
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars->o_empty[s]);
                }
#pragma unroll
                for (int h8 = 0; h8 < 4; ++h8) {
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t y = mul2(f2(o[16 * h8 + 2 * e], o[16 * h8 + 2 * e + 1]), f2(li, li));
                        zero = fma2(y, 0, zero);
                        float y0, y1;
                        unf2(y, y0, y1);
                        w[e] = pack2(y0, y1);
                    }
                    if (row_ok) {    // whole 32-byte sectors of the thread's own row
                        if (p.wide) {
                            store32(dst + c + 16 * h8, w);
                        } else {
                            *reinterpret_cast<uint4 *>(dst + c + 16 * h8) = make_uint4(w[0], w[1], w[2], w[3]);
                            *reinterpret_cast<uint4 *>(dst + c + 16 * h8 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
            float z0, z1;
            unf2(zero, z0, z1);
            bad = bad || (row_ok && z0 + z1 != 0.f);   // looked at after the last block
        }
        __syncwarp();                // the rows as their threads have stored them
        if (ok && __any_sync(0xffffffffu, bad)) redo_rows<DH>(p, s, quad, lane);
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 512);
}

template <int DH>
hcsa_status launch(const SwaArgs &a, cudaStream_t st) {
    using Sz = Sizes<DH>;
    static_assert(Sz::kSmem <= 232448 && sizeof(Bars<Sz::kStages>) + 16 <= 1024, "shared memory per CTA");
    static bool opted[64];
    if (!shared_opt_in((const void *)swa_tc_kernel<DH>, Sz::kSmem, opted)) return HCSA_ERR_CUDA;
    Args p;
    p.a = a;
    p.G = a.H / a.Hkv;
    p.tb = kRows / p.G;
    p.wide = ((uintptr_t)a.out & 31) == 0 && a.ld_out % 16 == 0;
    p.blocks = (uint32_t)((a.row1 - a.row0 + 2 * p.tb - 1) / (2 * p.tb));
    if ((int64_t)p.blocks * a.Hkv > INT32_MAX / 2) return HCSA_ERR_UNSUPPORTED;
    p.n_units = p.blocks * a.Hkv;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    CUtensorMap q, k, v, k16, v16;
    const uint64_t rows = a.row1, nkv = (uint64_t)a.Hkv * DH;   // tokens behind the row range are not read
    if (!make_tmap_bf16_3d(&q, a.q, DH, a.H, rows, DH * 2, a.ld_q * 2, 64, p.G, p.tb, true) ||
        !make_tmap_bf16_2d(&k, a.k, nkv, rows, a.ld_k * 2, 64, kKT, true) ||
        !make_tmap_bf16_2d(&v, a.v, nkv, rows, a.ld_v * 2, 64, kKT, true) ||
        !make_tmap_bf16_2d(&k16, a.k, nkv, rows, a.ld_k * 2, 64, kGran, true) ||
        !make_tmap_bf16_2d(&v16, a.v, nkv, rows, a.ld_v * 2, 64, kGran, true))
        return HCSA_ERR_CUDA;
    const unsigned sms = sm_grid(1), grid = p.n_units < sms ? p.n_units : sms;
    swa_tc_kernel<DH><<<grid, kThreads, Sz::kSmem, st>>>(q, k, v, k16, v16, p);
    count_launch();
    return check_launch();
}

}  // namespace

bool swa_tc_supported(const SwaArgs &a) {
    return a.dtype == HCSA_BF16 && (a.dh == 64 || a.dh == 128) && a.scale > 0.f && a.scale < 1e30f;
}

hcsa_status launch_swa_tc(const SwaArgs &a, cudaStream_t st) {
    return a.dh == 64 ? launch<64>(a, st) : launch<128>(a, st);
}

}  // namespace hcsa
