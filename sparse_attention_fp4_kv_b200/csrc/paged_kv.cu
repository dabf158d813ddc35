// FP4 append into pages, and the rows back in bf16.
//
// The quantization is kv_append.cu's own (kv_quant.cuh), the destination of a
// row comes from its sequence's page table. One thread per scale group, as in
// the contiguous append: a row of 512 channels is one warp, so its loads (32 B
// per lane), code stores (8 B) and scale stores (1 B) are coalesced, and the
// 32 lanes' table look-ups fall on one word.
#include "kv_quant.cuh"
#include "paged.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace csa2 {
namespace pkv {

constexpr int THREADS = 256;

// Row (b, i) and group g of work item gid; false when the row is to be skipped,
// else its row in the pool.
__device__ __forceinline__ bool locate(int64_t gid, int G, int B, int n, const int64_t *start,
                                       const int32_t *n_valid, const PagedKv &pk, int &g, int64_t &row,
                                       int64_t &cell) {
    row = gid / G;
    g = (int)(gid - row * G);
    const int64_t b = row / n;
    const int i = (int)(row - b * n);
    if (n_valid && i >= __ldg(n_valid + b)) return false;
    cell = paged_row(pk, b, __ldg(start + b) + i);
    return cell >= 0;
}

template <bool MX>
__global__ void __launch_bounds__(THREADS)
    append_kernel(const uint16_t *__restrict__ kv, int B, int n, int C, const int64_t *__restrict__ start,
                  const int32_t *__restrict__ n_valid, PagedKv pk, uint8_t *__restrict__ fp4,
                  uint8_t *__restrict__ sf) {
    constexpr int GC = MX ? 32 : 16;
    const int G = C / GC;
    const int64_t gid = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (gid >= (int64_t)B * n * G) return;
    int g;
    int64_t row, cell;
    if (!locate(gid, G, B, n, start, n_valid, pk, g, row, cell)) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(kv + row * C + (int64_t)g * GC);
    uint8_t *dst = fp4 + cell * (C / 2) + (int64_t)g * (GC / 2);
    uint32_t scode;
    if constexpr (MX) {
        const uint4 a[4] = {src[0], src[1], src[2], src[3]};
        *reinterpret_cast<uint4 *>(dst) = mxfp4_quant32(a, scode);
    } else {
        *reinterpret_cast<uint2 *>(dst) = fp4_quant16(src[0], src[1], scode);
    }
    sf[cell * G + g] = (uint8_t)scode;
}

// Eight codes -> eight bf16 values times the scale (exact: 2 + 4 significant bits).
__device__ __forceinline__ uint4 dequant8(uint32_t codes, float s) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t byte = codes >> (8 * j);
        const __nv_bfloat162 h =
            __floats2bfloat162_rn(e2m1_to_f32(byte & 15) * s, e2m1_to_f32((byte >> 4) & 15) * s);
        o[j] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool MX>
__global__ void __launch_bounds__(THREADS)
    gather_kernel(const uint8_t *__restrict__ fp4, const uint8_t *__restrict__ sf, PagedKv pk,
                  const int64_t *__restrict__ start, const int32_t *__restrict__ n_valid, int B, int n,
                  int C, uint16_t *__restrict__ out) {
    const int G = C / 16;  // 16 channels per thread in both formats
    const int64_t gid = (int64_t)blockIdx.x * THREADS + threadIdx.x;
    if (gid >= (int64_t)B * n * G) return;
    int g;
    int64_t row, cell;
    if (!locate(gid, G, B, n, start, n_valid, pk, g, row, cell)) return;
    const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(fp4 + cell * (C / 2) + (int64_t)g * 8));
    const float s = MX ? e8m0_to_f32(__ldg(sf + cell * (C / 32) + (g >> 1)))
                       : e4m3_to_f32(__ldg(sf + cell * G + g));
    uint4 *dst = reinterpret_cast<uint4 *>(out + row * C + (int64_t)g * 16);
    dst[0] = dequant8(codes.x, s);
    dst[1] = dequant8(codes.y, s);
}

int grid_of(int64_t items, dim3 &grid) {
    const int64_t blocks = (items + THREADS - 1) / THREADS;
    if (blocks > INT32_MAX) return CSA2_ERR_SHAPE;
    grid = dim3((unsigned)blocks);
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
    const int st = grid_of((int64_t)B * n * (C / GC), grid);
    if (st != CSA2_OK) return st;
    return launch_kernel(false, append_kernel<MX>, grid, dim3(THREADS), 0, (cudaStream_t)stream,
                         (const uint16_t *)kv, B, n, C, start, n_valid,
                         PagedKv{table, max_pages, page_size, n_pages}, fp4, sf);
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
    const int st = grid_of((int64_t)B * n * (C / 16), grid);
    if (st != CSA2_OK) return st;
    return launch_kernel(false, gather_kernel<MX>, grid, dim3(THREADS), 0, (cudaStream_t)stream, fp4, sf,
                         PagedKv{table, max_pages, page_size, n_pages}, start, n_valid, B, n, C,
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
