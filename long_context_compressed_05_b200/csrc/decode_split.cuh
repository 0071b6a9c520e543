// How a decode step over ragged paged sequences is split over CTAs, shared by its kernels.
//
// A unit is (sequence, key head, block of query heads); its work is the sequence's chunks of CT (16 or 32) tokens.  All
// units' chunks in order form one list that the CTAs share out in equal contiguous pieces, whatever the
// sequences' lengths; a CTA walks its piece unit by unit (segments).  A unit inside one piece is finished by
// its CTA; the others leave one partial per CTA (at most the piece's first and last segment: two slots), and
// a second kernel joins them in CTA order, so the result does not depend on timing.  Where no unit can have
// more than kDirectTokens tokens (a short window), every CTA takes one whole unit and nothing is joined.
#pragma once

#include "sliding.cuh"

namespace hcsa {

constexpr int kDirectTokens = 256;
// Chunks of a piece at least, so that a step over short sequences does not join more partials than it saves: 128 tokens, or
// 256 where FP8 chunks are 32 (taken at 16-token chunks, not measured again for 32).
constexpr int kMinShare = 8;

struct Split {
    int units_per_seq;              // key heads x head blocks
    int direct;                     // one CTA per unit
    int64_t *prefix;                // [B + 1] chunks before each sequence's units (unused when direct)
    float *ml;                      // [grid][2][heads][2]
    float *acc;                     // [grid][2][heads][dh]
};

struct Segment {
    int b, u;                       // sequence, unit within it
    int c0, c1, n;                  // chunks of the unit: this segment's, and all
};

__device__ __forceinline__ int64_t capacity_of(const DecodeArgs &a) { return (int64_t)a.c.max_pages * a.c.page; }

__device__ __forceinline__ int64_t share_of(int64_t total, int64_t grid) {
    const int64_t s = (total + grid - 1) / grid;
    return s < kMinShare ? kMinShare : s;
}

// Inclusive scan over the block (NT threads); every thread calls it.  Returns the thread's inclusive sum, total in *all.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *all, int64_t *sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) sh[warp] = v;
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += sh[i];
        sum += sh[i];
    }
    __syncthreads();
    *all = sum;
    return before + v;
}

// This CTA's piece: its first sequence, the offset of the piece in that sequence's units, and its length.
// CTA 0 also writes the prefix array for the joining kernel.
struct Piece {
    int b;
    int64_t off, len;
};
template <int NT, int CT>
__device__ __forceinline__ Piece piece_of(const DecodeArgs &a, const Split &s, int64_t *sh) {
    __shared__ int sh_b;
    __shared__ int64_t sh_off;
    int64_t total = 0, all;
    for (int base = 0; base < a.c.B; base += NT) {
        const int b = base + threadIdx.x;
        const int64_t v =
            b < a.c.B ? (int64_t)decode_keys<CT>(a.pos[b], a.window, a.sinks, capacity_of(a), a.c.status).n * s.units_per_seq : 0;
        const int64_t incl = block_scan<NT>(v, &all, sh);
        if (blockIdx.x == 0 && b < a.c.B) s.prefix[b] = total + incl - v;
        total += all;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) s.prefix[a.c.B] = total;
    const int64_t share = share_of(total, gridDim.x), start = share * blockIdx.x;
    Piece p{0, 0, 0};
    if (start >= total) return p;
    p.len = total - start < share ? total - start : share;
    int64_t run = 0;
    for (int base = 0; base < a.c.B && run <= start; base += NT) {
        const int b = base + threadIdx.x;
        const int64_t v =
            b < a.c.B ? (int64_t)decode_keys<CT>(a.pos[b], a.window, a.sinks, capacity_of(a), nullptr).n * s.units_per_seq : 0;
        const int64_t incl = run + block_scan<NT>(v, &all, sh);
        if (incl - v <= start && start < incl) {
            sh_b = b;
            sh_off = start - (incl - v);
        }
        run += all;
    }
    __syncthreads();
    p.b = sh_b;
    p.off = sh_off;
    return p;
}

size_t decode_split_bytes(int B, int grid, int heads, int dh);
Split make_split(const DecodeArgs &a, int units_per_seq, int heads, int grid);
// zero rows of empty slots and join the partials; heads: query heads per unit, grid: CTAs of the split kernel
hcsa_status launch_decode_join(const DecodeArgs &a, const Split &s, int heads, int grid, cudaStream_t st);
bool decode_direct(const DecodeArgs &a);

hcsa_status launch_decode_simt(const DecodeArgs &a, cudaStream_t st);
int decode_simt_heads(int dh);
bool decode_tc_supported(int dtype, int dh);
int decode_tc_heads();
int decode_tc_grid();
hcsa_status launch_decode_tc(const DecodeArgs &a, cudaStream_t st);

}  // namespace hcsa
