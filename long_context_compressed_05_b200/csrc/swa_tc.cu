// Sliding-window prefill attention on the tensor cores (tcgen05 + TMEM, TMA box loads): bf16, dh 64 or 128, any group of
// heads, window and first tokens.
//
// A block is two sub-tiles of 128 query rows of one key head: a row is a (token, head of the group) pair, a sub-tile
// holds floor(128 / G) tokens.  Both sub-tiles walk the same tiles of 128 key columns (the first tokens outside the
// window, padded to 16, then the tokens from the first row's window on; see block_keys) and share their loads.
//   S = Q K^T        128 x 128 fp32 in TMEM, one buffer per sub-tile
//   online softmax   a warpgroup per sub-tile, a thread per row (no exchange between threads); the running maximum is
//                    raised, and O rescaled in TMEM, only when a row's maximum grows by more than 2^8
//   O += P V         P (bf16) as the A operand in TMEM, written over S; V an MN-major B operand from shared memory
// The tensor core alternates between the sub-tiles (P V of one, then its next S), so one sub-tile's products run
// while the other's softmax does; the S of the next block is issued right behind the last P V of this one.
// Persistent CTAs take the blocks longest first, in a snake order over the CTAs.  Warps: 0 TMA, 1 MMA, 4..7 and 8..11
// softmax and output of sub-tile 0 and 1 (rows staged through shared memory a warp at a time, so that the stores are
// whole 128-byte lines).
//
// Per tile of 128 x 128 at dh 128 the products take 1024 cycles of the tensor core and the exponentials 1024 of
// the special-function unit: two equal bounds for a long window.
#include "sliding.cuh"
#include "tc_common.cuh"

namespace hcsa {

namespace {

constexpr int kRows = 128;           // query rows of a sub-tile
constexpr int kKT = 128;             // key columns of a tile
constexpr int kGran = 16;            // rows of the small TMA boxes: padding of the first tokens' columns
constexpr int kThreads = 384;
// Registers a thread: 168 at launch (384 threads), shared out anew as 72 for the TMA / MMA warpgroup and 208 for
// the two softmax warpgroups (128 x 72 + 256 x 208 <= 384 x 168)
constexpr int kRegsIssue = 72, kRegsSoftmax = 208;
constexpr uint32_t kColO = 256;      // TMEM: S (later P) of sub-tile s at 128 s, O at 256 + 128 s
constexpr float kSlack = 8.f;        // exp2 units

struct Args {
    SwaArgs a;
    int G, tb;                       // heads per key head, tokens per sub-tile
    uint32_t blocks, n_units;        // blocks of tokens, x key heads
    float scale_log2;
};

template <int DH> struct Sizes {
    static constexpr int kChunk = kRows * 128;              // 128 rows x 64 bf16
    static constexpr int kTile = DH / 64 * kChunk;          // Q, K or V tile
    static constexpr int kStages = DH == 128 ? 2 : 4;       // of K and of V
    static constexpr int kStaging = 8 * 4096;               // 32 rows x 128 bytes per softmax warp
    static constexpr int kSmem = 2 * kTile + 2 * kStages * kTile + kStaging + 2048;
};

template <int NST> struct Bars {
    uint64_t k_full[NST], k_empty[NST], v_full[NST], v_empty[NST];
    uint64_t q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2], drain;
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
// The issuing warp runs its loop with all lanes, so that addresses and descriptors stay in uniform registers; one
// elected lane (always the same) issues.  With a single active lane each product cost 120 cycles to issue.
// D[tmem] (+)= A[smem] B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc),
                 "r"(accumulate)
                 : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A's row i in lane i, two bf16 per 32-bit column
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t at, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(at), "l"(bdesc), "r"(idesc),
                 "r"(accumulate)
                 : "memory");
}
// mma_commit by the elected lane
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar))
                 : "memory");
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
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

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
swa_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_k16,
              const __grid_constant__ CUtensorMap tm_v16, const __grid_constant__ Args p) {
    using Sz = Sizes<DH>;
    constexpr int NST = Sz::kStages, NC = DH / 64;
    constexpr uint32_t kIdescS = tc::idesc_bf16(128, 128, false, false);
    constexpr uint32_t kIdescPV = tc::idesc_bf16(128, DH, false, true);
    const SwaArgs &a = p.a;
    extern __shared__ uint8_t smem_raw[];
    Bars<NST> *bars = reinterpret_cast<Bars<NST> *>(smem_raw);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 1);
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(tmem_slot + 4) + 1023) & ~uintptr_t(1023));
    uint8_t *staging = base + (2 + 2 * NST) * Sz::kTile;
    const uint32_t Qs = tc::smem_u32(base), Ks = Qs + 2 * Sz::kTile, Vs = Ks + NST * Sz::kTile;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            tc::mbar_init(&bars->k_full[i], 1);
            tc::mbar_init(&bars->k_empty[i], 1);
            tc::mbar_init(&bars->v_full[i], 1);
            tc::mbar_init(&bars->v_empty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc::mbar_init(&bars->q_full[s], 1);
            tc::mbar_init(&bars->q_empty[s], 1);
            tc::mbar_init(&bars->s_full[s], 1);
            tc::mbar_init(&bars->p_half[s], 4);
            tc::mbar_init(&bars->p_full[s], 4);
            tc::mbar_init(&bars->o_full[s], 1);
            tc::mbar_init(&bars->o_empty[s], 4);
        }
        tc::mbar_init(&bars->drain, 1);
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
        if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        if (lane == 0) {
            uint32_t it = 0, nq[2] = {0, 0}, nk = 0, nv = 0;   // tiles; loads issued
            auto load_q = [&](const Unit &x, int s) {
                if (x.c.hi(s) < 0) return;
                if (nq[s]) ok = ok && tc::mbar_wait(&bars->q_empty[s], (nq[s] - 1) & 1, a.status);
                if (!ok) return;
                tc::mbar_arrive_expect_tx(&bars->q_full[s], NC * 128 * p.tb * p.G);
                for (int c = 0; c < NC; ++c)
                    tc::tma_load_3d(Qs + s * Sz::kTile + c * Sz::kChunk, &tm_q, c * 64, x.g * p.G, x.first(s, p.tb),
                                    &bars->q_full[s]);
                ++nq[s];
            };
            auto load_kv = [&](const Unit &x, int i, bool v) {
                uint64_t *full = v ? bars->v_full : bars->k_full, *empty = v ? bars->v_empty : bars->k_empty;
                const int st = it % NST;
                if (it >= NST) ok = ok && tc::mbar_wait(&empty[st], (it / NST - 1) & 1, a.status);
                if (!ok) return;
                const uint32_t dst = (v ? Vs : Ks) + st * Sz::kTile;
                const int c0 = i * kKT;
                tc::mbar_arrive_expect_tx(&full[st], Sz::kTile);
                for (int c = 0; c < NC; ++c) {
                    const int x0 = x.g * DH + c * 64;
                    if (c0 >= x.c.pad) {
                        tc::tma_load_2d(dst + c * Sz::kChunk, v ? &tm_v : &tm_k, x0, x.w0 + c0 - x.c.pad, &full[st]);
                    } else {
                        for (int r = 0; r < kKT; r += kGran)
                            tc::tma_load_2d(dst + c * Sz::kChunk + r * 128, v ? &tm_v16 : &tm_k16, x0,
                                            c0 + r < x.c.pad ? c0 + r : x.w0 + c0 + r - x.c.pad, &full[st]);
                    }
                }
                ++(v ? nv : nk);
            };
            for (int k = 0; ok; ++k) {
                const int u = nth_unit(p, k);
                if (u < 0) break;
                const Unit x = unit_of(p, u);
                load_q(x, 0);
                for (int i = 0; i < x.c.n_tiles && ok; ++i, ++it) {
                    load_kv(x, i, false);
                    if (i == 0) load_q(x, 1);
                    if (ok) load_kv(x, i, true);
                }
            }
            // given up: the copies still in flight land (bounded waits) before the shared memory goes away
            if (!ok) {
                for (uint32_t n = nk > NST ? nk - NST : 0; n < nk; ++n)
                    tc::mbar_wait(&bars->k_full[n % NST], (n / NST) & 1, a.status);
                for (uint32_t n = nv > NST ? nv - NST : 0; n < nv; ++n)
                    tc::mbar_wait(&bars->v_full[n % NST], (n / NST) & 1, a.status);
                for (int s = 0; s < 2; ++s)
                    if (nq[s]) tc::mbar_wait(&bars->q_full[s], (nq[s] - 1) & 1, a.status);
            }
        }
        } else if (warp == 1) {
        // ---------------------------------------------------------- MMA issuer
        {
            uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};   // Q tiles, P tiles, blocks seen
            bool fresh[2] = {true, true};                             // no P V of the block yet
            struct Cursor { int k, i; uint32_t it; bool valid; Cols c; };
            auto start = [&](int k, uint32_t it) {
                Cursor c;
                const int u = nth_unit(p, k);
                c.valid = u >= 0;
                if (c.valid) c.c = unit_of(p, u).c;
                c.k = k;
                c.i = 0;
                c.it = it;
                return c;
            };
            // has the block a further tile for s?  Its last one is always active
            auto later = [&](const Cursor &c, int s) { return c.i < c.c.hi(s) / kKT; };
            auto active = [&](const Cursor &c, int s) { return c.c.active(s, c.i); };
            bool in[2] = {false, false};   // an S of the block has been issued
            const uint64_t q0 = tc::sdesc_sw128(Qs, 16, 1024), k0 = tc::sdesc_sw128(Ks, 16, 1024),
                           v0 = tc::sdesc_sw128(Vs, Sz::kChunk, 1024);
            auto issue_s = [&](const Cursor &c, int s) {
                const int st = c.it % NST;
                if (!in[s]) ok = ok && tc::mbar_wait(&bars->q_full[s], nq[s] & 1, a.status);
                ok = ok && tc::mbar_wait(&bars->k_full[st], (c.it / NST) & 1, a.status);
                if (!ok) return;
                tc::tc_fence_after();
                const uint64_t qd = q0 + s * (Sz::kTile >> 4), kd = k0 + st * (Sz::kTile >> 4);
#pragma unroll
                for (int k = 0; k < DH / 16; ++k) {
                    constexpr int kC = Sz::kChunk >> 4;
                    mma_ss(tmem + s * 128, qd + (k >> 2) * kC + 2 * (k & 3), kd + (k >> 2) * kC + 2 * (k & 3), kIdescS,
                                 k != 0 ? 1u : 0u);
                }
                commit(&bars->s_full[s]);
                in[s] = later(c, s);
                if (!in[s]) {        // the block's last S of this sub-tile
                    commit(&bars->q_empty[s]);
                    ++nq[s];
                }
            };
            auto issue_pv = [&](const Cursor &c, int s) {
                const int st = c.it % NST;
                ok = ok && tc::mbar_wait(&bars->v_full[st], (c.it / NST) & 1, a.status);
                if (fresh[s] && no[s]) ok = ok && tc::mbar_wait(&bars->o_empty[s], (no[s] - 1) & 1, a.status);
                const uint64_t vd = v0 + st * (Sz::kTile >> 4);
#pragma unroll
                for (int k = 0; k < kKT / 16; ++k) {
                    if (k == 0) ok = ok && tc::mbar_wait(&bars->p_half[s], np[s] & 1, a.status);
                    if (k == kKT / 32) ok = ok && tc::mbar_wait(&bars->p_full[s], np[s] & 1, a.status);
                    if (!ok) return;
                    if (k % (kKT / 32) == 0) tc::tc_fence_after();
                    mma_ts(tmem + kColO + s * 128, tmem + s * 128 + 8 * k, vd + 128 * k, kIdescPV,
                           !fresh[s] || k != 0 ? 1u : 0u);
                }
                ++np[s];
                fresh[s] = !later(c, s);
                if (fresh[s]) {
                    commit(&bars->o_full[s]);
                    ++no[s];
                }
            };
            Cursor cur = start(0, 0);
            if (cur.valid) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (active(cur, s)) issue_s(cur, s);
                if (ok) commit(&bars->k_empty[cur.it % NST]);
            }
            while (cur.valid && ok) {
                Cursor nxt = cur;
                ++nxt.it;
                if (++nxt.i == cur.c.n_tiles) nxt = start(cur.k + 1, cur.it + 1);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (active(cur, s)) issue_pv(cur, s);
                    if (ok && nxt.valid && active(nxt, s)) issue_s(nxt, s);
                }
                if (!ok) break;
                // K is waited for here too where no sub-tile uses it, so that its next load comes after this one
                if (nxt.valid && !active(nxt, 0) && !active(nxt, 1))
                    ok = tc::mbar_wait(&bars->k_full[nxt.it % NST], (nxt.it / NST) & 1, a.status);
                if (!active(cur, 0) && !active(cur, 1))
                    ok = ok && tc::mbar_wait(&bars->v_full[cur.it % NST], (cur.it / NST) & 1, a.status);
                if (nxt.valid) commit(&bars->k_empty[nxt.it % NST]);
                commit(&bars->v_empty[cur.it % NST]);
                cur = nxt;
            }
            if (!ok) {               // given up: the products in flight end (bounded wait) before their memory goes away
                commit(&bars->drain);
                tc::mbar_wait(&bars->drain, 0, a.status);
            }
        }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ---------------------------------------------------------- softmax + output (one warpgroup per sub-tile)
        const int s = (warp - 4) >> 2, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16), tS = lanes + s * 128, tO = lanes + kColO + s * 128;
        const int tl = r / p.G, hh = r - tl * p.G;
        uint8_t *stage = staging + (warp - 4) * 4096;
        uint32_t ns = 0, nu = 0;     // S tiles and blocks seen
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
            for (int i = 0; i < x.c.n_tiles; ++i) {
                if (!x.c.active(s, i)) continue;
                ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars->s_full[s], ns & 1, a.status));
                if (!ok) break;
                ++ns;
                tc::tc_fence_after();
                float v[kKT];
#pragma unroll
                for (int c = 0; c < kKT; c += 32) tc::tmem_ld32(tS + c, v + c);
                tc::tmem_ld_wait();
                const int c0 = i * kKT;
                const bool clean = c0 + kKT - 1 <= x.hi(ta) && (c0 >= x.lo(te, a.window) || c0 + kKT <= x.c.sk);
                if (!clean) {
#pragma unroll
                    for (int q = 0; q < kKT; q += 32) {
                        // bit c: column c0 + q + c is seen
                        auto upto = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
                        const int cg = c0 + q;
                        const uint32_t bits = upto(hi + 1 - cg) & (~upto(lo - cg) | upto(x.c.sk - cg));
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (!(bits >> c & 1)) v[q + c] = -INFINITY;
                    }
                }
                float mx[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) mx[c] = fmaxf(v[c], v[c + 8]);
#pragma unroll
                for (int c = 16; c < kKT; c += 16)
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = fmaxf(mx[e], fmaxf(v[c + e], v[c + e + 8]));
                float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
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
                const float ref = m == -INFINITY ? 0.f : m;   // a row that has seen no key yet: every weight 0
                const uint64_t sc2 = f2(p.scale_log2, p.scale_log2), ref2 = f2(-ref, -ref);
                uint64_t sum[4] = {0, 0, 0, 0};   // pairs of zeros
#pragma unroll
                for (int q = 0; q < kKT; q += 64) {
                    float w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float e0, e1;
                        unf2(fma2(f2(v[q + 2 * c], v[q + 2 * c + 1]), sc2, ref2), e0, e1);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        sum[c & 3] = add2(sum[c & 3], f2(e0, e1));
                        w[c] = __uint_as_float(pack2(e0, e1));
                    }
                    tc::tmem_st32(tS + q / 2, w);
                    tc::tmem_st_wait();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(q == 0 ? &bars->p_half[s] : &bars->p_full[s]);
                }
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
            const int64_t at = row_ok ? (int64_t)t * a.ld_out + (int64_t)(x.g * p.G + hh) * DH : -1;
            const float li = 1.f / l;
            float zero = 0.f;        // NaN once an output is not finite
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
                for (int g8 = 0; g8 < 8; ++g8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y0 = o[8 * g8 + 2 * e] * li, y1 = o[8 * g8 + 2 * e + 1] * li;
                        zero = fmaf(y0, 0.f, fmaf(y1, 0.f, zero));
                        w[e] = pack2(y0, y1);
                    }
                    *reinterpret_cast<uint4 *>(stage + tc::sw128_offset(lane, g8)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q) {   // four rows of 128 bytes at a time
                    const int row = 4 * q + (lane >> 3);
                    const int64_t to = __shfl_sync(0xffffffffu, at, row);
                    const uint4 w = *reinterpret_cast<const uint4 *>(stage + tc::sw128_offset(row, lane & 7));
                    if (to >= 0) *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.out + to + c + 8 * (lane & 7)) = w;
                }
                __syncwarp();
            }
            // rows that are not finite: by a value that they do not see? (the columns loaded for the block)
            for (unsigned bad = __ballot_sync(0xffffffffu, row_ok && zero != 0.f); bad; bad &= bad - 1) {
                const int row = quad * 32 + __ffs(bad) - 1, rt = ta + row / p.G;
                const int end = min(a.row1, x.w0 + x.c.n_tiles * kKT - x.c.pad);
                if (values_bad<__nv_bfloat16>(a, x.g, x.w0, (int64_t)rt - a.window + 1, lane) ||
                    values_bad<__nv_bfloat16>(a, x.g, rt + 1, end, lane) ||
                    (x.c.pad && values_bad<__nv_bfloat16>(a, x.g, x.c.sk, x.c.pad, lane)))
                    attend_row<__nv_bfloat16>(a, rt, x.g * p.G + row % p.G, lane);
            }
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 0) tc::tmem_free(tmem, 512);
}

template <int DH>
hcsa_status launch(const SwaArgs &a, cudaStream_t st) {
    using Sz = Sizes<DH>;
    static_assert(Sz::kSmem <= 232448 && sizeof(Bars<Sz::kStages>) + 16 <= 1024, "shared memory per CTA");
    if (cudaFuncSetAttribute(swa_tc_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sz::kSmem) != cudaSuccess)
        return HCSA_ERR_CUDA;
    Args p;
    p.a = a;
    p.G = a.H / a.Hkv;
    p.tb = kRows / p.G;
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
