// Paged key / value cache: new tokens' rows into the pages, in the storage type or as block-scaled FP8.
// Bandwidth- or launch-bound.  A block takes up to kRows rows: one thread per row finds where it goes (position, page,
// bounds), then the block copies the rows' 16-byte vectors.  A thread keeps its column (so its head, channel and
// addresses' strides are worked out once) and takes rows in turn, four in flight: with a flat index per vector the two
// divisions and the addresses were half of the FP8 kernel's instructions (8191 rows of 8 heads of 128, FP8, in a captured
// graph: 15.3 us against 13.0 to 13.9; about 21 a call where the host makes them one by one).  In bf16 8.7 us.
#include "sliding.cuh"

namespace hcsa {

namespace {

constexpr int kRows = 32, kThreads = 256;

// nv: 16-byte vectors of one row's heads (Hkv dh / VEC): vectors 0 .. nv - 1 of a row are k's, the next nv v's
template <typename S, bool FP8>
__global__ void __launch_bounds__(kThreads)
page_append_kernel(PageArgs a, int64_t rows, int per_block, int nv, int shift, const int32_t *pos, const int32_t *seq, const S *k,
                   int64_t ld_k, const S *v, int64_t ld_v) {
    constexpr int V = Traits<S>::VEC;
    __shared__ int sm_line[kRows];   // row of head 0 in the page arrays, -1: the row is skipped
    const int64_t r0 = (int64_t)blockIdx.x * per_block;
    const int n = rows - r0 < per_block ? (int)(rows - r0) : per_block;
    if (threadIdx.x < n) {
        const int64_t r = r0 + threadIdx.x;
        const int p = pos[r];
        const int64_t b = seq ? seq[r] : r;
        int line = -1;
        if (p >= 0 && b >= 0) {
            int id = -1;
            if (b < a.B && p < (int64_t)a.max_pages * a.page) id = a.table[b * a.max_pages + p / a.page];
            if (id < 0 || id >= a.n_pages) report(a.status, kStatusBounds);
            else line = id * a.Hkv * a.page + p % a.page;   // below 2^31 (checked on the host)
        }
        sm_line[threadIdx.x] = line;
    }
    // columns tx, tx + 2^shift, ... of rows ty, ty + 256 / 2^shift, ...
    const int tx = threadIdx.x & ((1 << shift) - 1), ty = threadIdx.x >> shift, step = kThreads >> shift;
    bool placed = false;
    for (int c0 = 0; c0 < 2 * nv; c0 += 1 << shift) {
        const int c = c0 + tx;
        const bool in = c < 2 * nv, is_v = c >= nv;
        const int at = (is_v ? c - nv : c) * V, g = in ? at / a.dh : 0, d = at - g * a.dh;
        const S *src = (is_v ? v + r0 * ld_v : k + r0 * ld_k) + at;
        const int64_t ld = is_v ? ld_v : ld_k;
        void *dst = is_v ? a.v_pages : a.k_pages;
        uint8_t *exps = (uint8_t *)dst + (int64_t)a.n_pages * a.Hkv * a.page * a.dh + d / 32;   // FP8
        for (int r = ty; r - ty < n; r += 4 * step) {   // the same turns for the whole block
            uint4 raw[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                raw[j] = make_uint4(0, 0, 0, 0);
                if (in && r + j * step < n) raw[j] = __ldg(reinterpret_cast<const uint4 *>(src + (r + j * step) * ld));
            }
            if (!placed) {
                __syncthreads();     // the rows' places, looked up while the first loads run
                placed = true;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int line = in && r + j * step < n ? sm_line[r + j * step] : -1;
                const int64_t to = (int64_t)line + (int64_t)g * a.page;
                if constexpr (!FP8) {
                    if (line >= 0) *reinterpret_cast<uint4 *>((S *)dst + to * a.dh + d) = raw[j];
                } else {
                    // the four threads of a 32-channel block are consecutive lanes of one row; the whole warp shuffles
                    float x[V];
                    const S *e = reinterpret_cast<const S *>(&raw[j]);
#pragma unroll
                    for (int q = 0; q < V; ++q) x[q] = (float)e[q];
                    float amax = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
                    for (int q = 2; q < V; q += 2) amax = fmaxf(amax, fmaxf(fabsf(x[q]), fabsf(x[q + 1])));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                    if (line >= 0) {
                        const int ex = page_exponent(amax);
                        *reinterpret_cast<uint2 *>((uint8_t *)dst + to * a.dh + d) = codes_of(x, ex);
                        if ((d & 31) == 0) exps[to * (a.dh / 32)] = (uint8_t)(int8_t)ex;
                    }
                }
            }
        }
    }
}

}  // namespace

hcsa_status launch_page_append(const PageArgs &a, int64_t rows, const int32_t *pos, const int32_t *seq, const void *k,
                               int64_t ld_k, const void *v, int64_t ld_v, cudaStream_t st) {
    if (rows == 0) return HCSA_OK;
    const int64_t nv64 = (int64_t)a.Hkv * a.dh / (a.dtype == HCSA_BF16 ? 8 : 4);
    if (nv64 > 1 << 23) return HCSA_ERR_UNSUPPORTED;
    const int nv = (int)nv64;
    // rows per block: about two thousand vectors (FP8 as above: 13.0 us; a thousand 14.5, four thousand 14.0), fewer where the
    // blocks would not fill the GPU
    int64_t per = 2048 / (2 * nv);
    const int64_t spread = rows / (4 * sm_grid(1));
    if (per > spread) per = spread;
    if (per > kRows) per = kRows;
    if (per < 1) per = 1;
    const int64_t blocks = (rows + per - 1) / per;
    if (blocks > INT32_MAX) return HCSA_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)blocks, threads = kThreads;
    const int rpb = (int)per;
    int shift = 3;                   // a row's vectors rounded up to a power of two, up to the block
    while (shift < 8 && (1 << shift) < 2 * nv) ++shift;
    if (a.dtype == HCSA_F32)
        page_append_kernel<float, false><<<grid, threads, 0, st>>>(a, rows, rpb, nv, shift, pos, seq, (const float *)k, ld_k,
                                                               (const float *)v, ld_v);
    else if (a.lowprec)
        page_append_kernel<__nv_bfloat16, true><<<grid, threads, 0, st>>>(a, rows, rpb, nv, shift, pos, seq, (const __nv_bfloat16 *)k,
                                                                      ld_k, (const __nv_bfloat16 *)v, ld_v);
    else
        page_append_kernel<__nv_bfloat16, false><<<grid, threads, 0, st>>>(a, rows, rpb, nv, shift, pos, seq, (const __nv_bfloat16 *)k,
                                                                       ld_k, (const __nv_bfloat16 *)v, ld_v);
    count_launch();
    return check_launch();
}

}  // namespace hcsa
