// Attention of one new token over a paged FP4 cache: the call, the kernel for
// E4M3 scales (paged_attn.cuh), and the joining of a pair's parts.
#include "paged_attn.cuh"

namespace csa2 {

int paged_attn_wait_flag(bool clear) { return read_device_flag(pa::g_paged_attn_error, clear); }

int pa::launch_paged_attn_fp4(const Args &a, int nh, int G, cudaStream_t s) { return launch_attn<false>(a, nh, G, s); }

namespace pa {

// Joins the parts that the CTAs of a split (sequence, head group) pair left:
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. Block (pair, y) takes
// `per` heads; its threads are columns of four channels times groups of parts, so
// that many parts' loads are in flight. Pairs without a key get zeros here, pairs
// within one CTA are already finished. Block (0, 0) also sets the error word.
constexpr int JT = 512;
constexpr int MAX_PARTS = 1024;  // CTAs of the attention kernel
__global__ void __launch_bounds__(JT) join_kernel(const Args a, int NH, int pitch, int G, int per, int *err) {
    __shared__ float weight[MAX_PARTS];
    __shared__ float4 acc[JT];
    __shared__ float red[2][JT / 32];
    grid_dep_wait();
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int any = 0;
        for (int i = tid; i < G; i += JT) any |= a.flags[i];
        any = __syncthreads_or(any);
        if (tid == 0) *err = any != 0;
    }
    const int b = blockIdx.x / a.groups, g = blockIdx.x % a.groups;
    const int64_t T = a.prefix[a.B] * a.groups, p0 = a.prefix[b], tiles = a.prefix[b + 1] - p0;
    const int64_t t0 = p0 * a.groups + g * tiles;
    const int sharers = sharing(T, G);
    const int lo = tiles ? owner_of(t0, T, sharers) : 0, hi = tiles ? owner_of(t0 + tiles - 1, T, sharers) : 0;
    if (tiles && lo == hi) return;
    const int n = hi - lo + 1;
    // the part of the first CTA: its second segment unless its share starts here
    const int slot0 = 2 * lo + (tiles && share_begin(lo, T, sharers) != t0 ? 1 : 0);
    auto slot = [&](int i) { return i == 0 ? slot0 : 2 * (lo + i); };
    const int cols = a.C / 4, col = tid % cols, grp = tid / cols, groups = JT / cols;
    for (int y = 0; y < per; y++) {
        const int hh = blockIdx.y * per + y, h = g * NH + hh;
        if (hh >= NH || h >= a.Hq) break;
        uint2 *out = reinterpret_cast<uint2 *>(a.out + ((int64_t)b * a.Hq + h) * a.C);
        float *lse = a.lse ? a.lse + (int64_t)b * a.Hq + h : nullptr;
        if (!tiles) {
            if (tid < cols) out[tid] = make_uint2(0, 0);
            if (tid == 0 && lse) *lse = -INFINITY;
            continue;
        }
        float m = REF_NONE;
        for (int i = tid; i < n; i += JT) m = fmaxf(m, a.part_ml[((int64_t)slot(i) * NH + hh) * 2]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        if ((tid & 31) == 0) red[0][tid >> 5] = m;
        __syncthreads();
        for (int i = 0; i < JT / 32; i++) m = fmaxf(m, red[0][i]);
        float sum = 0.0f;
        for (int i = tid; i < n; i += JT) {
            const float *ml = a.part_ml + ((int64_t)slot(i) * NH + hh) * 2;
            const float wt = ex2(ml[0] - m);
            weight[i] = wt;
            sum += wt * ml[1];
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if ((tid & 31) == 0) red[1][tid >> 5] = sum;
        __syncthreads();
        sum = 0.0f;
        for (int i = 0; i < JT / 32; i++) sum += red[1][i];
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (grp < groups) {
            const float *o = a.part_o + (int64_t)hh * pitch + 4 * col;
#pragma unroll 8
            for (int i = grp; i < n; i += groups) {
                const float4 x = *reinterpret_cast<const float4 *>(o + (int64_t)slot(i) * NH * pitch);
                const float wt = weight[i];
                v.x += wt * x.x;
                v.y += wt * x.y;
                v.z += wt * x.z;
                v.w += wt * x.w;
            }
        }
        acc[tid] = v;
        __syncthreads();
        if (tid < cols) {
            for (int i = 1; i < groups; i++) {
                const float4 x = acc[i * cols + tid];
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
            }
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            out[tid] = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        }
        if (tid == 0 && lse) *lse = sum != 0.0f ? (m + log2f(sum)) * LN2 : -INFINITY;
        __syncthreads();
    }
}

// Heads of one group: the smallest MMA width that holds them, 64 at most.
int group_heads(int Hq) { return Hq <= 16 ? 16 : Hq <= 32 ? 32 : 64; }

constexpr size_t up(size_t x) { return (x + 255) / 256 * 256; }
// Workspace: the error word, the CTAs' flags, the tiles before each sequence,
// and two parts per CTA.
struct Ws {
    int *err, *flags;
    int64_t *prefix;
    float *ml, *o;
    size_t bytes;
};
Ws layout(void *base, int B, int Hq, int C, int G) {
    const int nh = group_heads(Hq), pitch = (C + 127) / 128 * 128;
    char *p = static_cast<char *>(base);
    size_t off = 0;
    Ws w;
    auto take = [&](size_t bytes) {
        char *q = p + off;
        off += up(bytes);
        return q;
    };
    w.err = reinterpret_cast<int *>(take(sizeof(int)));
    w.flags = reinterpret_cast<int *>(take(sizeof(int) * (size_t)G));
    w.prefix = reinterpret_cast<int64_t *>(take(sizeof(int64_t) * ((size_t)B + 1)));
    w.ml = reinterpret_cast<float *>(take(sizeof(float) * 2 * 2 * (size_t)G * nh));
    w.o = reinterpret_cast<float *>(take(sizeof(float) * 2 * (size_t)G * nh * pitch));
    w.bytes = off;
    return w;
}

// One CTA per SM: the shared memory of one leaves no room for a second.
int grid_ctas() {
    const int n = num_sms();
    return n < MAX_PARTS ? n : MAX_PARTS;
}

int decode(bool mx, const void *q, const uint8_t *fp4, const uint8_t *sf, const int32_t *table, int max_pages,
           int page_size, int n_pages, const int64_t *ctx_len, int64_t n_win, int64_t n_sink, int B, int Hq,
           int C, float scale, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (B != 0 && (!q || !fp4 || !sf || !table || !ctx_len || !out)) return CSA2_ERR_NULL;
    if (B < 0 || Hq < 1 || Hq > 256 || C < 32 || C > 512 || C % 32 ||
        !paged_shape_ok(max_pages, page_size, n_pages))
        return CSA2_ERR_SHAPE;
    const int64_t cap = (int64_t)max_pages * page_size;
    if (cap > INT32_MAX) return CSA2_ERR_SHAPE;
    if (n_win < 0 || n_sink < 0) return CSA2_ERR_RANGE;
    if (!aligned(q, 16) || !aligned(fp4, 16) || !aligned(out, 8) || (!mx && !aligned(sf, 4))) return CSA2_ERR_ALIGN;
    if (B == 0) return CSA2_OK;
    const int G = grid_ctas(), nh = group_heads(Hq), groups = (Hq + nh - 1) / nh;
    if ((int64_t)B * groups > INT32_MAX) return CSA2_ERR_SHAPE;
    const Ws w = layout(ws, B, Hq, C, G);
    if (!ws || ws_bytes < w.bytes) return CSA2_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return CSA2_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const Args a{(const uint16_t *)q, fp4, sf, PagedKv{table, max_pages, page_size, n_pages}, ctx_len,
                 (int)(n_win < cap ? n_win : cap), (int)(n_sink < cap ? n_sink : cap), (int)cap, fast_div(page_size), B, Hq, C, groups, scale, (uint16_t *)out, lse, w.flags, w.prefix, w.ml, w.o};
    const int st = mx ? launch_paged_attn_mxfp4(a, nh, G, s) : launch_paged_attn_fp4(a, nh, G, s);
    if (st != CSA2_OK) return st;
    // one head per block until there are a few blocks per SM
    const int pairs = B * groups;
    int blocks = 4 * G / pairs;
    blocks = blocks < 1 ? 1 : blocks > nh ? nh : blocks;
    const int per = (nh + blocks - 1) / blocks;
    return launch_kernel(true, join_kernel, dim3((unsigned)pairs, (unsigned)((nh + per - 1) / per)), dim3(JT), 0,
                         s, a, nh, (C + 127) / 128 * 128, G, per, w.err);
}

}  // namespace pa
}  // namespace csa2

extern "C" size_t csa2_paged_attn_workspace_size(int B, int Hq, int C) {
    if (B < 1 || Hq < 1 || C < 1) return 0;
    return csa2::pa::layout(nullptr, B, Hq, C, csa2::pa::grid_ctas()).bytes;
}

extern "C" int csa2_paged_attn_decode(const void *q_bf16, const uint8_t *kv_fp4, const uint8_t *kv_sf,
                                      const int32_t *page_table, int max_pages, int page_size, int n_pages,
                                      const int64_t *ctx_len, int64_t n_win, int64_t n_sink, int B, int Hq,
                                      int C, float softmax_scale, void *out_bf16, float *lse, void *ws,
                                      size_t ws_bytes, void *stream) {
    return csa2::pa::decode(false, q_bf16, kv_fp4, kv_sf, page_table, max_pages, page_size, n_pages, ctx_len,
                            n_win, n_sink, B, Hq, C, softmax_scale, out_bf16, lse, ws, ws_bytes, stream);
}

extern "C" int csa2_paged_attn_decode_mxfp4(const void *q_bf16, const uint8_t *kv_fp4, const uint8_t *kv_sf,
                                            const int32_t *page_table, int max_pages, int page_size,
                                            int n_pages, const int64_t *ctx_len, int64_t n_win,
                                            int64_t n_sink, int B, int Hq, int C, float softmax_scale,
                                            void *out_bf16, float *lse, void *ws, size_t ws_bytes,
                                            void *stream) {
    return csa2::pa::decode(true, q_bf16, kv_fp4, kv_sf, page_table, max_pages, page_size, n_pages, ctx_len,
                            n_win, n_sink, B, Hq, C, softmax_scale, out_bf16, lse, ws, ws_bytes, stream);
}
