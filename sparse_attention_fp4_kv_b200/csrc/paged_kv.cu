// FP4 append into pages, and the rows back in bf16.
//
// The quantization is kv_append.cu's own (kv_quant.cuh), the destination of a
// row comes from its sequence's page table. One lane per scale group, as in
// the contiguous append: a row of 512 channels is one warp, so its loads (32 B
// per lane), code stores (8 B) and scale stores (1 B) are coalesced, and the
// 32 lanes' table look-ups fall on one word. 262,144 rows of 512 (344 MB each way,
// 52.5 us at the copy rate): MXFP4 append 62.4 us and read-back 64 to 65 are bound by
// memory, by loads in flight and CTAs that have work. The FP4 append, 92.0 us, is
// bound by instructions: 2.4 times those of the MXFP4 form (a scale, its reciprocal, a
// row look-up and a 64-bit division per 16 channels instead of 32, and a product, two
// clamps and two integer steps per channel), 80 % of the issue slots and 37 % of
// DRAM's rate. 65,536 rows: 23.3 us (MXFP4 15.8), read-back 17.3.
#include "fp4_rows.cuh"
#include "kv_quant.cuh"
#include "paged.cuh"

namespace csa2 {
namespace pkv {

constexpr int THREADS = 128;
constexpr int BATCH = 2;  // groups of a thread, all loaded before the first is stored
constexpr int PER_CTA = THREADS * BATCH;
constexpr int MOST = 2 * (2048 / THREADS);  // CTAs per SM of a padded call

// A CTA takes PER_CTA groups of its sequence. With n_valid most rows may be
// padding, and CTAs that only find that out are what a large call spends its time
// on: beyond two waves of CTAs a padded call walks its groups instead, PER_CTA at
// a time and `step` apart (8 chunks of up to 8192 rows, 8527 in all: append and
// read-back 12.4 us, with a CTA for every group 15.2; without padding the walk
// costs, 65,536 rows 38.0 against 36.4).
struct Span {
    int b;                     // sequence
    int64_t first, end, step;  // groups of the sequence: this CTA's first, and behind the last valid row's
};
__device__ __forceinline__ Span span_of(int G, int n, const int32_t *n_valid, int blocks) {
    Span s;
    s.step = (int64_t)blocks * PER_CTA;
    s.b = blockIdx.x / blocks;
    s.first = (int64_t)(blockIdx.x - s.b * blocks) * PER_CTA;
    int rows = n;
    if (n_valid) {
        const int v = __ldg(n_valid + s.b);
        rows = v < n ? v : n;
    }
    s.end = (int64_t)rows * G;
    return s;
}
template <bool MX, bool WALK>
__global__ void __launch_bounds__(THREADS)
    append_kernel(const uint16_t *__restrict__ kv, int n, int C, const int64_t *__restrict__ start,
                  const int32_t *__restrict__ n_valid, PagedKv pk, int blocks, uint8_t *__restrict__ fp4,
                  uint8_t *__restrict__ sf) {
    constexpr int GC = MX ? 32 : 16, LOADS = GC / 8;
    const int G = C / GC;
    grid_dep_wait();
    grid_dep_launch();
    const Span s = span_of(G, n, n_valid, blocks);
    if (s.first >= s.end) return;
    const int64_t pos0 = __ldg(start + s.b);
    for (int64_t first = s.first; first < s.end; first += s.step) {
        uint4 x[BATCH][LOADS];
        int64_t cell[BATCH];
        int g[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; k++) {
            const int64_t at = first + k * THREADS + threadIdx.x;
            cell[k] = -1;
            if (at >= s.end) continue;
            const int64_t i = at / G;
            g[k] = (int)(at - i * G);
            const uint4 *src = reinterpret_cast<const uint4 *>(kv + ((int64_t)s.b * n + i) * C + g[k] * GC);
#pragma unroll
            for (int j = 0; j < LOADS; j++) x[k][j] = ld_stream_v4(src + j);
            cell[k] = paged_row(pk, s.b, pos0 + i);
        }
#pragma unroll
        for (int k = 0; k < BATCH; k++) {
            if (cell[k] < 0) continue;
            uint8_t *dst = fp4 + cell[k] * (C / 2) + g[k] * (GC / 2);
            uint32_t scode;
            if constexpr (MX)
                *reinterpret_cast<uint4 *>(dst) = mxfp4_quant32(x[k], scode);
            else
                *reinterpret_cast<uint2 *>(dst) = fp4_quant16(x[k][0], x[k][1], scode);
            sf[cell[k] * G + g[k]] = (uint8_t)scode;
        }
        if constexpr (!WALK) break;
    }
}

template <bool MX, bool WALK>
__global__ void __launch_bounds__(THREADS)
    gather_kernel(const uint8_t *__restrict__ fp4, const uint8_t *__restrict__ sf, PagedKv pk,
                  const int64_t *__restrict__ start, const int32_t *__restrict__ n_valid, int n, int C, int blocks,
                  uint16_t *__restrict__ out) {
    const int G = C / 16;  // 16 channels per thread in both formats
    grid_dep_wait();
    grid_dep_launch();
    const Span s = span_of(G, n, n_valid, blocks);
    if (s.first >= s.end) return;
    const int64_t pos0 = __ldg(start + s.b);
    for (int64_t first = s.first; first < s.end; first += s.step) {
        uint2 codes[BATCH];
        uint32_t scale[BATCH];
        int64_t to[BATCH];  // group of out, < 0: none
#pragma unroll
        for (int k = 0; k < BATCH; k++) {
            const int64_t at = first + k * THREADS + threadIdx.x;
            to[k] = -1;
            if (at >= s.end) continue;
            const int64_t i = at / G;
            const int g = (int)(at - i * G);
            const int64_t cell = paged_row(pk, s.b, pos0 + i);
            if (cell < 0) continue;
            to[k] = ((int64_t)s.b * n + i) * G + g;
            codes[k] = __ldg(reinterpret_cast<const uint2 *>(fp4 + cell * (C / 2) + g * 8));
            scale[k] = MX ? __ldg(sf + cell * (C / 32) + (g >> 1)) : __ldg(sf + cell * G + g);
        }
#pragma unroll
        for (int k = 0; k < BATCH; k++) {
            if (to[k] < 0) continue;
            const MxScale s2 = MX ? mx_scale(scale[k]) : e4m3_scale(scale[k]);
            uint4 *dst = reinterpret_cast<uint4 *>(out + to[k] * 16);
            dst[0] = rows_bf16(codes[k].x, s2);
            dst[1] = rows_bf16(codes[k].y, s2);
        }
        if constexpr (!WALK) break;
    }
}

// CTAs per sequence, the grid, and whether they walk.
int grid_of(int B, int64_t groups, bool padded, int &blocks, dim3 &grid, bool &walk) {
    int64_t per = (groups + PER_CTA - 1) / PER_CTA;
    const int64_t most = ((int64_t)MOST * num_sms() + B - 1) / B;
    walk = padded && per > most;
    if (walk) per = most;
    if (per * B > INT32_MAX) return CSA2_ERR_SHAPE;
    blocks = (int)per;
    grid = dim3((unsigned)(per * B));
    return CSA2_OK;
}

template <bool MX>
int append(const void *kv, int B, int n, int C, const int64_t *start, const int32_t *n_valid,
           const int32_t *table, int max_pages, int page_size, int n_pages, uint8_t *fp4, uint8_t *sf,
           void *stream) {
    constexpr int GC = MX ? 32 : 16;
    if (B != 0 && n != 0 && (!kv || !start || !table || !fp4 || !sf)) return CSA2_ERR_NULL;
    if (B < 0 || n < 0 || C < GC || C > 8192 || C % GC || !paged_shape_ok(max_pages, page_size, n_pages))
        return CSA2_ERR_SHAPE;
    if (!aligned(kv, 16) || !aligned(fp4, MX ? 16 : 8)) return CSA2_ERR_ALIGN;
    if ((int64_t)B * n == 0) return CSA2_OK;
    dim3 grid;
    int blocks;
    bool walk;
    const int st = grid_of(B, (int64_t)n * (C / GC), n_valid != nullptr, blocks, grid, walk);
    if (st != CSA2_OK) return st;
    return launch_kernel(true, walk ? append_kernel<MX, true> : append_kernel<MX, false>, grid, dim3(THREADS), 0, (cudaStream_t)stream,
                         (const uint16_t *)kv, n, C, start, n_valid,
                         PagedKv{table, max_pages, page_size, n_pages}, blocks, fp4, sf);
}

template <bool MX>
int gather(const uint8_t *fp4, const uint8_t *sf, const int32_t *table, int max_pages, int page_size,
           int n_pages, const int64_t *start, const int32_t *n_valid, int B, int n, int C, void *out,
           void *stream) {
    constexpr int GC = MX ? 32 : 16;
    if (B != 0 && n != 0 && (!fp4 || !sf || !table || !start || !out)) return CSA2_ERR_NULL;
    if (B < 0 || n < 0 || C < GC || C > 8192 || C % GC || !paged_shape_ok(max_pages, page_size, n_pages))
        return CSA2_ERR_SHAPE;
    if (!aligned(out, 16) || !aligned(fp4, 8)) return CSA2_ERR_ALIGN;
    if ((int64_t)B * n == 0) return CSA2_OK;
    dim3 grid;
    int blocks;
    bool walk;
    const int st = grid_of(B, (int64_t)n * (C / 16), n_valid != nullptr, blocks, grid, walk);
    if (st != CSA2_OK) return st;
    return launch_kernel(true, walk ? gather_kernel<MX, true> : gather_kernel<MX, false>, grid, dim3(THREADS), 0, (cudaStream_t)stream, fp4, sf,
                         PagedKv{table, max_pages, page_size, n_pages}, start, n_valid, n, C, blocks,
                         (uint16_t *)out);
}

}  // namespace pkv
}  // namespace csa2

extern "C" int csa2_paged_kv_append_fp4(const void *kv_bf16, int B, int n_new, int C,
                                        const int64_t *start_pos, const int32_t *n_valid,
                                        const int32_t *page_table, int max_pages, int page_size,
                                        int n_pages, uint8_t *kv_fp4, uint8_t *kv_sf, void *stream) {
    return csa2::pkv::append<false>(kv_bf16, B, n_new, C, start_pos, n_valid, page_table, max_pages,
                                    page_size, n_pages, kv_fp4, kv_sf, stream);
}

extern "C" int csa2_paged_kv_append_mxfp4(const void *kv_bf16, int B, int n_new, int C,
                                          const int64_t *start_pos, const int32_t *n_valid,
                                          const int32_t *page_table, int max_pages, int page_size,
                                          int n_pages, uint8_t *kv_fp4, uint8_t *kv_sf, void *stream) {
    return csa2::pkv::append<true>(kv_bf16, B, n_new, C, start_pos, n_valid, page_table, max_pages,
                                   page_size, n_pages, kv_fp4, kv_sf, stream);
}

extern "C" int csa2_paged_kv_gather_fp4(const uint8_t *kv_fp4, const uint8_t *kv_sf,
                                        const int32_t *page_table, int max_pages, int page_size,
                                        int n_pages, const int64_t *start_pos, const int32_t *n_valid,
                                        int B, int n, int C, void *out_bf16, void *stream) {
    return csa2::pkv::gather<false>(kv_fp4, kv_sf, page_table, max_pages, page_size, n_pages, start_pos,
                                    n_valid, B, n, C, out_bf16, stream);
}

extern "C" int csa2_paged_kv_gather_mxfp4(const uint8_t *kv_fp4, const uint8_t *kv_sf,
                                          const int32_t *page_table, int max_pages, int page_size,
                                          int n_pages, const int64_t *start_pos,
                                          const int32_t *n_valid, int B, int n, int C, void *out_bf16,
                                          void *stream) {
    return csa2::pkv::gather<true>(kv_fp4, kv_sf, page_table, max_pages, page_size, n_pages, start_pos,
                                   n_valid, B, n, C, out_bf16, stream);
}
