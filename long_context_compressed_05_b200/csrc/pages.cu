// Paged key / value cache: new tokens' rows into the pages, in the storage type or as block-scaled FP8.
// Bandwidth- or launch-bound: one thread per 16-byte vector of the sources, no shared state.
#include "sliding.cuh"

namespace hcsa {

namespace {

// nv: 16-byte vectors of one row's heads (Hkv dh / VEC); threads 0 .. nv - 1 of a row take k, the rest v
template <typename S, bool FP8>
__global__ void __launch_bounds__(256) page_append_kernel(PageArgs a, int64_t rows, int nv, const int32_t *pos,
                                                          const int32_t *seq, const S *k, int64_t ld_k, const S *v,
                                                          int64_t ld_v) {
    constexpr int V = Traits<S>::VEC;
    const int64_t total = rows * 2 * nv;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / (2 * nv);
        int c = (int)(i - r * 2 * nv);
        const bool is_v = c >= nv;
        if (is_v) c -= nv;
        const int p = pos[r];
        const int64_t b = seq ? seq[r] : r;
        if (p < 0 || b < 0) continue;
        if (b >= a.B || p >= (int64_t)a.max_pages * a.page) {
            report(a.status, kStatusBounds);
            continue;
        }
        const int id = a.table[b * a.max_pages + p / a.page];
        if (id < 0 || id >= a.n_pages) {
            report(a.status, kStatusBounds);
            continue;
        }
        const int g = c * V / a.dh, d = c * V - g * a.dh;
        const int64_t line = ((int64_t)id * a.Hkv + g) * a.page + p % a.page;
        const uint4 raw = __ldg(reinterpret_cast<const uint4 *>((is_v ? v + r * ld_v : k + r * ld_k) + c * V));
        void *dst = is_v ? a.v_pages : a.k_pages;
        if constexpr (!FP8) {
            *reinterpret_cast<uint4 *>((S *)dst + line * a.dh + d) = raw;
        } else {
            // the four threads of a 32-channel block are four consecutive lanes: 2 nv and the block size are
            // multiples of 4, so they share the row and leave the loop together
            float x[V];
            const S *e = reinterpret_cast<const S *>(&raw);
#pragma unroll
            for (int q = 0; q < V; ++q) x[q] = (float)e[q];
            const int ex = page_exponent(lp::block_amax(x));
            uint8_t *codes = (uint8_t *)dst;
            *reinterpret_cast<uint2 *>(codes + line * a.dh + d) = codes_of(x, ex);
            if ((d & 31) == 0)
                ((int8_t *)codes)[(int64_t)a.n_pages * a.Hkv * a.page * a.dh + line * (a.dh / 32) + d / 32] = (int8_t)ex;
        }
    }
}

}  // namespace

hcsa_status launch_page_append(const PageArgs &a, int64_t rows, const int32_t *pos, const int32_t *seq, const void *k,
                               int64_t ld_k, const void *v, int64_t ld_v, cudaStream_t st) {
    if (rows == 0) return HCSA_OK;
    const int nv = a.Hkv * a.dh / (a.dtype == HCSA_BF16 ? 8 : 4);
    const int64_t blocks = (rows * 2 * nv + 255) / 256;
    const unsigned grid = (unsigned)(blocks < (1 << 30) ? blocks : (1 << 30));
    if (a.dtype == HCSA_F32)
        page_append_kernel<float, false><<<grid, 256, 0, st>>>(a, rows, nv, pos, seq, (const float *)k, ld_k,
                                                               (const float *)v, ld_v);
    else if (a.lowprec)
        page_append_kernel<__nv_bfloat16, true><<<grid, 256, 0, st>>>(a, rows, nv, pos, seq, (const __nv_bfloat16 *)k,
                                                                      ld_k, (const __nv_bfloat16 *)v, ld_v);
    else
        page_append_kernel<__nv_bfloat16, false><<<grid, 256, 0, st>>>(a, rows, nv, pos, seq, (const __nv_bfloat16 *)k,
                                                                       ld_k, (const __nv_bfloat16 *)v, ld_v);
    count_launch();
    return check_launch();
}

}  // namespace hcsa
