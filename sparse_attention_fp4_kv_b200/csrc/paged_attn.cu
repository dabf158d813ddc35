// Attention of one new token over a paged FP4 cache.
//
// out = sum_j exp(s_j - m) row_j / sum_j exp(s_j - m), one pass over the keys
// with the running maximum m and sum of each head in fp32. One CTA takes eight
// heads of a sequence, a warp one head; tiles of 32 keys are dequantized to
// shared memory once for the eight.
#include "paged.cuh"

#include <cuda_bf16.h>

namespace csa2 {
namespace pa {

constexpr int TK = 32, WARPS = 8, THREADS = WARPS * 32, MAX_C = 512;

struct Args {
    const uint16_t *q;
    const uint8_t *fp4, *sf;
    PagedKv pk;
    const int64_t *ctx_len;
    int64_t win, sink;
    int B, Hq, C;
    float scale;
    uint16_t *out;
    float *lse;
    int *err;  // the call's error word
};

template <bool MX>
__global__ void __launch_bounds__(THREADS) simple_kernel(const Args a) {
    extern __shared__ float sm[];
    const int pitch = a.C + 1;
    float *tile = sm;                 // [TK][C + 1]
    float *qs = sm + TK * pitch;      // [WARPS][C]
    float *ps = qs + WARPS * a.C;     // [WARPS][TK]
    __shared__ int ok[TK];
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.err = 0;
    const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.x * WARPS + warp;
    int64_t n = a.ctx_len[b];
    const int64_t cap = (int64_t)a.pk.max_pages * a.pk.page_size;
    if (n > cap) n = cap;
    if (n < 0) n = 0;
    int64_t ns = 0, w0 = 0;
    if (a.win > 0) {
        ns = a.sink < n ? a.sink : n;
        w0 = n - a.win > ns ? n - a.win : ns;
    }
    const int64_t nvis = ns + n - w0;
    if (h < a.Hq)
        for (int c = lane; c < a.C; c += 32)
            qs[warp * a.C + c] = __uint_as_float((uint32_t)a.q[((int64_t)b * a.Hq + h) * a.C + c] << 16);
    float m = -INFINITY, l = 0.0f, o[MAX_C / 32];
#pragma unroll
    for (int i = 0; i < MAX_C / 32; i++) o[i] = 0.0f;
    for (int64_t j0 = 0; j0 < nvis; j0 += TK) {
        __syncthreads();
        for (int i = threadIdx.x; i < TK * (a.C / 2); i += THREADS) {
            const int r = i / (a.C / 2), cb = i - r * (a.C / 2);
            const int64_t j = j0 + r;
            const int64_t row = j < nvis ? paged_row(a.pk, b, j < ns ? j : w0 + j - ns) : -1;
            float lo = 0.0f, hi = 0.0f;
            if (row >= 0) {
                const uint32_t byte = a.fp4[row * (a.C / 2) + cb];
                const float s = MX ? e8m0_to_f32(a.sf[row * (a.C / 32) + cb / 16])
                                   : e4m3_to_f32(a.sf[row * (a.C / 16) + cb / 8]);
                lo = e2m1_to_f32(byte & 15) * s;
                hi = e2m1_to_f32(byte >> 4) * s;
            }
            tile[r * pitch + 2 * cb] = lo;
            tile[r * pitch + 2 * cb + 1] = hi;
            if (cb == 0) ok[r] = row >= 0;
        }
        __syncthreads();
        if (h >= a.Hq) continue;
        float x = 0.0f;
        for (int c = 0; c < a.C; c++) x += qs[warp * a.C + c] * tile[lane * pitch + c];
        x = ok[lane] ? x * a.scale : -INFINITY;
        float mt = x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
        if (mt == -INFINITY) continue;
        const float m_new = fmaxf(m, mt);
        const float alpha = expf(m - m_new), p = expf(x - m_new);
        float sum = p;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * alpha + sum;
        m = m_new;
        ps[warp * TK + lane] = p;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < MAX_C / 32; i++) {
            if (i * 32 >= a.C) break;
            float v = o[i] * alpha;
            for (int r = 0; r < TK; r++) v += ps[warp * TK + r] * tile[r * pitch + i * 32 + lane];
            o[i] = v;
        }
        __syncwarp();
    }
    if (h >= a.Hq) return;
#pragma unroll
    for (int i = 0; i < MAX_C / 32; i++) {
        if (i * 32 >= a.C) break;
        const __nv_bfloat16 v = __float2bfloat16_rn(l != 0.0f ? o[i] / l : 0.0f);
        a.out[((int64_t)b * a.Hq + h) * a.C + i * 32 + lane] = *reinterpret_cast<const uint16_t *>(&v);
    }
    if (a.lse && lane == 0) a.lse[(int64_t)b * a.Hq + h] = l != 0.0f ? m + logf(l) : -INFINITY;
}

template <bool MX>
int decode(const void *q, const uint8_t *fp4, const uint8_t *sf, const int32_t *table, int max_pages,
           int page_size, int n_pages, const int64_t *ctx_len, int64_t n_win, int64_t n_sink, int B, int Hq,
           int C, float scale, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (B != 0 && (!q || !fp4 || !sf || !table || !ctx_len || !out)) return CSA2_ERR_NULL;
    if (B < 0 || Hq < 1 || Hq > 256 || C < 32 || C > MAX_C || C % 32 ||
        !paged_shape_ok(max_pages, page_size, n_pages))
        return CSA2_ERR_SHAPE;
    if (n_win < 0 || n_sink < 0) return CSA2_ERR_RANGE;
    if (!aligned(q, 16) || !aligned(fp4, 16) || (!MX && !aligned(sf, 4))) return CSA2_ERR_ALIGN;
    if (B == 0) return CSA2_OK;
    if (!ws || ws_bytes < csa2_paged_attn_workspace_size(B, Hq, C)) return CSA2_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return CSA2_ERR_ALIGN;
    static PerDevice smem_set;
    const size_t smem = sizeof(float) * ((size_t)TK * (C + 1) + (size_t)WARPS * (C + TK));
    if (!set_smem_limit_once(smem_set, simple_kernel<MX>, 100 * 1024)) return CSA2_ERR_CUDA;
    const Args a{(const uint16_t *)q, fp4, sf, PagedKv{table, max_pages, page_size, n_pages}, ctx_len,
                 n_win, n_sink, B, Hq, C, scale, (uint16_t *)out, lse, (int *)ws};
    return launch_kernel(false, simple_kernel<MX>, dim3((unsigned)(Hq + WARPS - 1) / WARPS, (unsigned)B),
                         dim3(THREADS), smem, (cudaStream_t)stream, a);
}

}  // namespace pa
}  // namespace csa2

extern "C" size_t csa2_paged_attn_workspace_size(int B, int Hq, int C) {
    if (B < 1 || Hq < 1 || C < 1) return 0;
    return 256;
}

extern "C" int csa2_paged_attn_decode(const void *q_bf16, const uint8_t *kv_fp4, const uint8_t *kv_sf,
                                      const int32_t *page_table, int max_pages, int page_size, int n_pages,
                                      const int64_t *ctx_len, int64_t n_win, int64_t n_sink, int B, int Hq,
                                      int C, float softmax_scale, void *out_bf16, float *lse, void *ws,
                                      size_t ws_bytes, void *stream) {
    return csa2::pa::decode<false>(q_bf16, kv_fp4, kv_sf, page_table, max_pages, page_size, n_pages, ctx_len,
                                   n_win, n_sink, B, Hq, C, softmax_scale, out_bf16, lse, ws, ws_bytes,
                                   stream);
}

extern "C" int csa2_paged_attn_decode_mxfp4(const void *q_bf16, const uint8_t *kv_fp4, const uint8_t *kv_sf,
                                            const int32_t *page_table, int max_pages, int page_size,
                                            int n_pages, const int64_t *ctx_len, int64_t n_win,
                                            int64_t n_sink, int B, int Hq, int C, float softmax_scale,
                                            void *out_bf16, float *lse, void *ws, size_t ws_bytes,
                                            void *stream) {
    return csa2::pa::decode<true>(q_bf16, kv_fp4, kv_sf, page_table, max_pages, page_size, n_pages, ctx_len,
                                  n_win, n_sink, B, Hq, C, softmax_scale, out_bf16, lse, ws, ws_bytes,
                                  stream);
}
