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
// Per tile of 128 x 128 at dh 128 the products take 1024 cycles of the tensor core and the exponentials 1024 of
// the special-function unit: two equal bounds for a long window.  What holds it above them is the chain of a
// sub-tile (S, softmax, P V, next S), of which TMEM has room for two.  Measured at 8192 tokens, 32 heads over 8, dh 128,
// causal: 409 us (1345 TFLOP/s).  What was tried there: P in one part 462; parts of 64 + 64 462, four of 32 479; two
// threads per row 466; two S buffers of 64 columns 458 (the narrow products are bound by shared memory); a quarter of
// the exponentials by a polynomial on the FMA pipe 441; one issuing warp for both sub-tiles 497.  A window of 128 (65536
// tokens, 64 heads over 8, dh 128: 680 us) is bound by the same chain: two tiles a block, then the output.  These are at
// 1965 MHz; seconds of such calls run at the power limit, 1500 to 1660 MHz (480 and 820 us).
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

// Rows of sub-tile s, lanes [32 quad, 32 quad + 32), of this CTA's blocks that came out non-finite by a value that they do
// not see, over exactly their keys.  By the warp that has stored them, once it has handed over its last block: nothing
// waits for it any more.  (A row of a long sequence takes as long as it has keys; the pipeline's waits are bounded.)
template <int DH>
__device__ __noinline__ void redo_rows(const Args &p, int s, int quad, int lane) {
    const SwaArgs &a = p.a;
    for (int k = 0;; ++k) {
        const int u = nth_unit(p, k);
        if (u < 0) break;
        const Unit x = unit_of(p, u);
        const int behind = min(a.row1, x.w0 + x.c.n_tiles * kKT - x.c.pad);   // tokens loaded for the block
        for (int r = 32 * quad; r < 32 * quad + 32; ++r) {
            const int tl = r / p.G, t = x.first(s, p.tb) + tl, h = x.g * p.G + r - tl * p.G;
            if (tl >= p.tb || t > x.last(s, p.tb)) break;
            const __nv_bfloat16 *o = (const __nv_bfloat16 *)a.out + (int64_t)t * a.ld_out + (int64_t)h * DH;
            bool fine = true;
            for (int d = lane; d < DH; d += 32) fine = fine && fabsf((float)o[d]) < INFINITY;
            if (__all_sync(0xffffffffu, fine)) continue;
            if ((values_bad<__nv_bfloat16>(a, x.g, x.w0, (int64_t)t - a.window + 1, lane) ||
                 values_bad<__nv_bfloat16>(a, x.g, t + 1, behind, lane) ||
                 (x.c.pad && values_bad<__nv_bfloat16>(a, x.g, x.c.sk, x.c.pad, lane))) &&
                !row_explained<__nv_bfloat16>(a, t, h, lane, 0, DH))
                attend_row<__nv_bfloat16>(a, t, h, lane, 0, DH);
        }
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
