// Attention of one new token over a paged FP4 cache: the call, the kernel for
// E4M3 scales (paged_attn.cuh), and the joining of a pair's parts.
#include "paged_attn.cuh"

namespace csa2 {

int paged_attn_wait_flag(bool clear) { return read_device_flag(pa::g_paged_attn_error, clear); }

int pa::launch_paged_attn_fp4(const Args &a, int nh, int G, cudaStream_t s) { return launch_attn<false>(a, nh, G, s); }

namespace pa {

// Joins the parts that the CTAs of a split (sequence, head group) pair left:
// out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i. A warp takes 128 channels of
// one head, four per lane, and 32 parts at a time: lane i reads part i's (m, l),
// the weights go round by shuffles; the first parts' O are on the way before the
// weights are known. A chain of loads, each as long as L2 takes: WIDE, the JW warps
// of a block share one such piece of work and take parts in turn, else each has its
// own. Pairs without a key get zeros here, pairs within one CTA are already finished.
// Block 0 also sets the error word.
constexpr int EARLY = 4;         // parts
constexpr int MAX_CTAS = 1024;   // of the attention kernel
template <int JW, bool WIDE>
__global__ void __launch_bounds__(JW * 32) join_kernel(const Args a, int NH, int pitch, int G, int chunks, int work, int *err) {
    __shared__ float4 acc_s[JW][32];
    __shared__ float2 ml_s[JW];
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0) {
        int any = 0;
        for (int i = threadIdx.x; i < G; i += JW * 32) any |= a.flags[i];
        any = __syncthreads_or(any);
        if (threadIdx.x == 0) *err = any != 0;
    }
    // work item: (pair, head of the group, chunk of 128 channels)
    const int item = WIDE ? blockIdx.x : blockIdx.x * JW + warp;
    if (item >= work) return;
    const int chunk = item % chunks, hh = item / chunks % NH, pair = item / chunks / NH;
    const int b = pair / a.groups, g = pair % a.groups, h = g * NH + hh, c = 128 * chunk + 4 * lane;
    if (h >= a.Hq) return;
    const int p0 = a.prefix[b], tiles = a.prefix[b + 1] - p0;
    uint2 *out = reinterpret_cast<uint2 *>(a.out + ((int64_t)b * a.Hq + h) * a.C + c);
    float *lse = a.lse && chunk == 0 && lane == 0 ? a.lse + (int64_t)b * a.Hq + h : nullptr;
    if (tiles == 0) {
        if ((!WIDE || warp == 0) && c < a.C) *out = make_uint2(0, 0);
        if ((!WIDE || warp == 0) && lse) *lse = -INFINITY;
        return;
    }
    const Shares shares(a.prefix[a.B] * a.groups, G);
    const int t0 = p0 * a.groups + g * tiles, lo = shares.owner(t0), hi = shares.owner(t0 + tiles - 1);
    if (lo == hi) return;
    const int n = hi - lo + 1;
    // the part of the first CTA: its second segment unless its share starts here
    const int slot0 = 2 * lo + (shares.begin(lo) != t0 ? 1 : 0);
    auto slot = [&](int i) { return i == 0 ? slot0 : 2 * (lo + i); };
    float m = REF_NONE, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int step = WIDE ? JW : 1, first = WIDE ? warp : 0;  // this warp's parts: first, first + step, ...
    for (int i0 = first; i0 < n; i0 += 32 * step) {
        const int count = (n - i0 + step - 1) / step < 32 ? (n - i0 + step - 1) / step : 32;
        const float *po = a.part_o + (int64_t)hh * pitch + c;
        float4 x[EARLY];  // asked for before the weights are known
#pragma unroll
        for (int j = 0; j < EARLY; j++) {
            x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (j < count) x[j] = *reinterpret_cast<const float4 *>(po + (int64_t)slot(i0 + j * step) * NH * pitch);
        }
        const int mine = i0 + lane * step;
        float2 ml = make_float2(REF_NONE, 0.0f);
        if (mine < n) ml = *reinterpret_cast<const float2 *>(a.part_ml + ((int64_t)slot(mine) * NH + hh) * 2);
        float top = fmaxf(m, ml.x);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float old = ex2(m - top), wt = ex2(ml.x - top);
        float sum = wt * ml.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        l = l * old + sum;
        o = make_float4(o.x * old, o.y * old, o.z * old, o.w * old);
        m = top;
#pragma unroll
        for (int j = 0; j < EARLY; j++) {
            const float w = __shfl_sync(0xffffffffu, wt, j);
            o.x += w * x[j].x;
            o.y += w * x[j].y;
            o.z += w * x[j].z;
            o.w += w * x[j].w;
        }
#pragma unroll 8
        for (int j = EARLY; j < count; j++) {
            const float w = __shfl_sync(0xffffffffu, wt, j);
            const float4 y = *reinterpret_cast<const float4 *>(po + (int64_t)slot(i0 + j * step) * NH * pitch);
            o.x += w * y.x;
            o.y += w * y.y;
            o.z += w * y.z;
            o.w += w * y.w;
        }
    }
    if constexpr (WIDE) {
        acc_s[warp][lane] = o;
        if (lane == 0) ml_s[warp] = make_float2(m, l);
        __syncthreads();
        if (warp > 0) return;
        float top = ml_s[0].x;
#pragma unroll
        for (int i = 1; i < JW; i++) top = fmaxf(top, ml_s[i].x);
        l = 0.0f;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < JW; i++) {
            const float w = ex2(ml_s[i].x - top);
            const float4 x = acc_s[i][lane];
            l += w * ml_s[i].y;
            o.x += w * x.x;
            o.y += w * x.y;
            o.z += w * x.z;
            o.w += w * x.w;
        }
        m = top;
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    if (c < a.C) *out = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (lse) *lse = l != 0.0f ? (m + log2f(l)) * LN2 : -INFINITY;
}

// Heads of one group: the smallest MMA width that holds them, 64 at most.
int group_heads(int Hq) { return Hq <= 16 ? 16 : Hq <= 32 ? 32 : 64; }

constexpr size_t up(size_t x) { return (x + 255) / 256 * 256; }
// Workspace: the error word, the CTAs' flags, the tiles before each sequence,
// and two parts per CTA.
struct Ws {
    int *err, *flags;
    int *prefix;
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
    w.prefix = reinterpret_cast<int *>(take(sizeof(int) * ((size_t)B + 1)));
    w.ml = reinterpret_cast<float *>(take(sizeof(float) * 2 * 2 * (size_t)G * nh));
    w.o = reinterpret_cast<float *>(take(sizeof(float) * 2 * (size_t)G * nh * pitch));
    w.bytes = off;
    return w;
}

// One CTA per SM: the shared memory of one leaves no room for a second.
int grid_ctas() {
    const int n = num_sms();
    return n < MAX_CTAS ? n : MAX_CTAS;
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
    const int pitch = (C + 127) / 128 * 128, chunks = pitch / 128;
    const int64_t work = (int64_t)B * groups * nh * chunks;
    // the kernels count tiles in 32 bits
    if (work > INT32_MAX || (int64_t)B * groups * (cap / TK + 1) > INT32_MAX) return CSA2_ERR_SHAPE;
    const Ws w = layout(ws, B, Hq, C, G);
    if (!ws || ws_bytes < w.bytes) return CSA2_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return CSA2_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const Args a{(const uint16_t *)q, fp4, sf, PagedKv{table, max_pages, page_size, n_pages}, ctx_len,
                 (int)(n_win < cap ? n_win : cap), (int)(n_sink < cap ? n_sink : cap), (int)cap,
                 fast_div(page_size), B, Hq, C, groups, scale, (uint16_t *)out, lse, w.flags, w.prefix, w.ml,
                 w.o};
    const int st = mx ? launch_paged_attn_mxfp4(a, nh, G, s) : launch_paged_attn_fp4(a, nh, G, s);
    if (st != CSA2_OK) return st;
    // Blocks of four warps fit beside an attention CTA and wait there for it. Up to
    // 16 pieces of work per SM a block shares one. With 24 parts or more to a pair
    // sixteen warps share it (attention and join, one sequence of 9000, 64 heads of
    // 512: 18.0 us with 16 warps, 20.8 with 8, 23.5 with 4; 8 sequences of 1000: 22.4
    // with 8, 18.3 with 4).
    auto join = [&](auto kernel, int warps, int blocks) {
        return launch_kernel(true, kernel, dim3((unsigned)blocks), dim3(warps * 32), 0, s, a, nh, pitch, G, chunks,
                             (int)work, w.err);
    };
    if (work > 16 * G) return join(join_kernel<4, false>, 4, (int)((work + 3) / 4));
    if (B * groups <= G / 24) return join(join_kernel<16, true>, 16, (int)work);
    return join(join_kernel<4, true>, 4, (int)work);
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
