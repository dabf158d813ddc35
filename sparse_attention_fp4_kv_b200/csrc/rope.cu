// Rotary positions of queries, cache rows and attention outputs.
//
// y = R(a) x per channel pair, a = pos * inv_freq. The angle of a far position
// (1M tokens x 1 radian) needs more bits than fp32 has, so its turns
// pos * inv_freq / 2pi are taken in fp64, reduced to [-1/2, 1/2] there, and only
// the reduced angle goes to the fp32 sincospi. Two fp64 products and one sincospi
// per (token, pair) of a CTA's tile serve all its heads.
//
// Bound by memory: each element is read once and written once. A CTA takes a
// tile of rows (one row = one head of one token), 16 bytes per thread and
// access; its cos/sin table goes to shared memory while its first loads are in
// flight. 4096 x 64 x 512 fp32 (1.07 GB): 161 us, 6.7 TB/s; 69,632 rows of 512 bf16
// (143 MB): 25.6 us, 5.6 TB/s; 4 tokens x 64 heads: 2.5 us. In place, 64 channels
// of 512: the 69,632 rows 20.8 us (18 MB, 2.8 us at the copy rate; what
// bounds it was not looked into), 4096 x 64 rows 16.9 in bf16 (67 MB), 24.6 in fp32 (134 MB).
#include "common.cuh"

#include <cuda_bf16.h>

namespace csa2 {
namespace rope {

constexpr int THREADS = 256;
constexpr int BATCH = 4;          // 16-byte accesses in flight per thread
constexpr int MAX_TABLE = 4096;   // (token, pair) entries of a CTA's table

struct Args {
    const void *x;
    void *out;
    const int64_t *pos;
    const double *freq;
    int64_t T;
    int H, D, start, rot;
    float sign, gain;       // sign of the sine, mscale
    int64_t xt, xh, ot, oh; // strides in elements
    int tt, hh;             // tile: tokens x heads
    int htiles;             // ceil(H / hh)
    int nrot, ncopy;        // rotated and copied items of a row
    uint32_t m_rot, m_copy, m_hh;  // magic numbers for / nrot, / ncopy and / hh
};

// n / d for n, d < 2^16 with m = ceil(2^32 / d) (m = 0: d = 1)
__device__ __forceinline__ uint32_t fast_div(uint32_t n, uint32_t m) { return m ? __umulhi(n, m) : n; }

__device__ __forceinline__ float ld1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld1(const float *p) { return *p; }
__device__ __forceinline__ void st1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void st1(float *p, float v) { *p = v; }

template <typename E>
__device__ __forceinline__ void unpack(uint4 w, float (&v)[16 / sizeof(E)]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = bf16_lo(u[i]);
            v[2 * i + 1] = bf16_hi(u[i]);
        }
    }
}
template <typename E>
__device__ __forceinline__ uint4 pack(const float (&v)[16 / sizeof(E)]) {
    uint32_t u[4];
    if constexpr (sizeof(E) == 4) {
#pragma unroll
        for (int i = 0; i < 4; i++) u[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float2 rotate(float u, float v, float2 cs) {
    return make_float2(u * cs.x - v * cs.y, v * cs.x + u * cs.y);
}

// cos and sin (times mscale) of the tile's tokens: table[t * pairs + i].
__device__ __forceinline__ void fill_table(const Args &a, int64_t t0, float2 *table) {
    const int pairs = a.rot / 2;
    for (int i = threadIdx.x; i < a.tt * pairs; i += THREADS) {
        const int t = i / pairs;
        if (t0 + t >= a.T) break;
        const double turns =
            (double)a.pos[t0 + t] * (a.freq[i - t * pairs] * 0.15915494309189533577);
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        table[i] = make_float2(c * a.gain, s * a.gain * a.sign);
    }
}

// Items of a row, 16 bytes (N channels) each: the copied pieces first, then the
// rotated ones. In the half layout a rotated item is two pieces, N channels of
// either half; they have a loop of their own, because their registers in the copies'
// loop cost occupancy (36 us for 69,632 rows of 512 channels with 64 rotated, at 75
// registers; the floor is 22).
template <typename E, bool HALF>
__global__ void __launch_bounds__(THREADS) vec_kernel(const Args a) {
    constexpr int N = 16 / sizeof(E);
    extern __shared__ float2 table[];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t0 = (int64_t)(blockIdx.x / a.htiles) * a.tt;
    const int h0 = (int)(blockIdx.x % a.htiles) * a.hh;
    const int rows = a.tt * a.hh;
    const E *x = static_cast<const E *>(a.x);
    E *out = static_cast<E *>(a.out);
    bool filled = false;

    const int copies = rows * a.ncopy;
    for (int base = 0; base < copies; base += THREADS * BATCH) {
        uint4 w[BATCH];
        int64_t to[BATCH];  // < 0: no item
#pragma unroll
        for (int k = 0; k < BATCH; k++) {
            const int i = base + k * THREADS + (int)threadIdx.x;
            const int row = (int)fast_div((uint32_t)i, a.m_copy);
            const int t = (int)fast_div((uint32_t)row, a.m_hh), h = h0 + row - t * a.hh;
            int c = (i - row * a.ncopy) * N;
            if (c >= a.start) c += a.rot;
            const bool in = i < copies && t0 + t < a.T && h < a.H;
            to[k] = in ? (t0 + t) * a.ot + (int64_t)h * a.oh + c : -1;
            if (in) w[k] = ld_stream_v4(x + (t0 + t) * a.xt + (int64_t)h * a.xh + c);
        }
        if (!filled) {  // while the first loads are in flight
            fill_table(a, t0, table);
            filled = true;
        }
#pragma unroll
        for (int k = 0; k < BATCH; k++)
            if (to[k] >= 0) *reinterpret_cast<uint4 *>(out + to[k]) = w[k];
    }
    if (!filled) fill_table(a, t0, table);
    __syncthreads();

    constexpr int RB = HALF ? 2 : BATCH;
    const int turns = rows * a.nrot;
    for (int base = 0; base < turns; base += THREADS * RB) {
        uint4 w[RB], w2[HALF ? RB : 1];
        int64_t to[RB];
        int entry[RB];  // table entry of the first pair
#pragma unroll
        for (int k = 0; k < RB; k++) {
            const int i = base + k * THREADS + (int)threadIdx.x;
            const int row = (int)fast_div((uint32_t)i, a.m_rot);
            const int t = (int)fast_div((uint32_t)row, a.m_hh), h = h0 + row - t * a.hh;
            const int piece = i - row * a.nrot, c = a.start + piece * N;
            const bool in = i < turns && t0 + t < a.T && h < a.H;
            to[k] = in ? (t0 + t) * a.ot + (int64_t)h * a.oh + c : -1;
            entry[k] = t * (a.rot / 2) + (HALF ? piece * N : piece * (N / 2));
            if (in) {
                const E *src = x + (t0 + t) * a.xt + (int64_t)h * a.xh + c;
                w[k] = *reinterpret_cast<const uint4 *>(src);
                if constexpr (HALF) w2[k] = *reinterpret_cast<const uint4 *>(src + a.rot / 2);
            }
        }
#pragma unroll
        for (int k = 0; k < RB; k++) {
            if (to[k] < 0) continue;
            const float2 *cs = table + entry[k];
            float u[N];
            unpack<E>(w[k], u);
            if constexpr (HALF) {
                float v[N];
                unpack<E>(w2[k], v);
#pragma unroll
                for (int j = 0; j < N; j++) {
                    const float2 r = rotate(u[j], v[j], cs[j]);
                    u[j] = r.x;
                    v[j] = r.y;
                }
                *reinterpret_cast<uint4 *>(out + to[k] + a.rot / 2) = pack<E>(v);
            } else {
#pragma unroll
                for (int j = 0; j < N; j += 2) {
                    const float2 r = rotate(u[j], u[j + 1], cs[j / 2]);
                    u[j] = r.x;
                    u[j + 1] = r.y;
                }
            }
            *reinterpret_cast<uint4 *>(out + to[k]) = pack<E>(u);
        }
    }
}

// Any alignment, stride and offset: an item is one pair or one copied channel.
template <typename E, bool HALF>
__global__ void __launch_bounds__(THREADS) scalar_kernel(const Args a) {
    extern __shared__ float2 table[];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t0 = (int64_t)(blockIdx.x / a.htiles) * a.tt;
    const int h0 = (int)(blockIdx.x % a.htiles) * a.hh;
    const int per_row = a.nrot + a.ncopy, items = a.tt * a.hh * per_row;
    fill_table(a, t0, table);
    __syncthreads();
    for (int i = threadIdx.x; i < items; i += THREADS) {
        const int row = i / per_row, piece = i - row * per_row;
        const int t = row / a.hh, h = h0 + row - t * a.hh;
        if (t0 + t >= a.T || h >= a.H) continue;
        const E *x = static_cast<const E *>(a.x) + (t0 + t) * a.xt + (int64_t)h * a.xh;
        E *out = static_cast<E *>(a.out) + (t0 + t) * a.ot + (int64_t)h * a.oh;
        if (piece < a.nrot) {
            const int u = a.start + (HALF ? piece : 2 * piece), v = u + (HALF ? a.rot / 2 : 1);
            const float2 r = rotate(ld1(x + u), ld1(x + v), table[t * (a.rot / 2) + piece]);
            st1(out + u, r.x);
            st1(out + v, r.y);
        } else {
            int c = piece - a.nrot;
            if (c >= a.start) c += a.rot;
            out[c] = x[c];
        }
    }
}

__global__ void freqs_kernel(int pairs, double theta, int scaling, double factor, double lo, double hi,
                             double *out) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= pairs) return;
    const double f = pow(theta, -(double)i / pairs);
    double r = 0.0;  // share of the stretched frequency
    if (scaling == CSA2_ROPE_LINEAR) r = 1.0;
    if (scaling == CSA2_ROPE_YARN) r = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
    out[i] = f * (1.0 - r) + f / factor * r;
}

inline uint32_t magic(int d) { return d == 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); }

template <typename E>
int launch(Args a, bool half, cudaStream_t s) {
    constexpr int N = 16 / sizeof(E);
    const bool in_place = a.x == a.out;
    // 16-byte accesses where every row and every part of it starts on 16 bytes
    const bool vec = aligned(a.x, 16) && aligned(a.out, 16) && a.xt % N == 0 && a.ot % N == 0 &&
                     (a.H == 1 || (a.xh % N == 0 && a.oh % N == 0)) && a.start % N == 0 &&
                     (half ? a.rot / 2 : a.rot) % N == 0 && a.D % N == 0;
    const int rest = in_place ? 0 : a.D - a.rot;
    a.nrot = vec ? (half ? a.rot / 2 / N : a.rot / N) : a.rot / 2;
    a.ncopy = vec ? rest / N : rest;
    // rows of a tile: two batches of 16-byte accesses per thread
    int want = 2 * BATCH * THREADS / (a.nrot + a.ncopy);
    // fewer where a small call would leave SMs idle (4 tokens x 64 heads of 512: 3.1 us
    // with 8 CTAs of 32 rows, 2.4 with one row a CTA)
    const int64_t spread = a.T * a.H / (2 * num_sms());
    if (spread < want) want = (int)spread;
    const int rows = want < 1 ? 1 : want;
    if (rows >= a.H) {
        a.hh = a.H;
        a.tt = rows / a.H;
        const int most = MAX_TABLE / (a.rot / 2);
        if (a.tt > most) a.tt = most;
        if (a.tt > a.T) a.tt = (int)a.T;
    } else {
        a.hh = rows;
        a.tt = 1;
    }
    a.htiles = (a.H + a.hh - 1) / a.hh;
    a.m_rot = magic(a.nrot);
    a.m_copy = a.ncopy ? magic(a.ncopy) : 0;
    a.m_hh = magic(a.hh);
    const int64_t blocks = ((a.T + a.tt - 1) / a.tt) * a.htiles;
    if (blocks > INT32_MAX) return CSA2_ERR_SHAPE;
    const size_t smem = sizeof(float2) * (size_t)a.tt * (a.rot / 2);
    const dim3 grid((unsigned)blocks), block(THREADS);
    if (vec) {  // a tile has at most 2 BATCH THREADS + D / N < 2^16 items: fast_div holds
        if (half) return launch_kernel(true, vec_kernel<E, true>, grid, block, smem, s, a);
        return launch_kernel(true, vec_kernel<E, false>, grid, block, smem, s, a);
    }
    if (half) return launch_kernel(true, scalar_kernel<E, true>, grid, block, smem, s, a);
    return launch_kernel(true, scalar_kernel<E, false>, grid, block, smem, s, a);
}

}  // namespace rope
}  // namespace csa2

extern "C" int csa2_rope(const void *x, void *out, int dtype, const int64_t *pos,
                         const double *inv_freq, int64_t T, int H, int D, int rot_start, int rot_dim,
                         int layout, int inverse, float mscale, int64_t x_tok_stride,
                         int64_t x_head_stride, int64_t out_tok_stride, int64_t out_head_stride,
                         void *stream) {
    using namespace csa2;
    if (T != 0 && (!x || !out || !pos || !inv_freq)) return CSA2_ERR_NULL;
    if (dtype != CSA2_BF16 && dtype != CSA2_F32) return CSA2_ERR_RANGE;
    if (layout != CSA2_ROPE_INTERLEAVED && layout != CSA2_ROPE_HALF) return CSA2_ERR_RANGE;
    if (T < 0 || H < 1 || D < 2 || D > 65536 || rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 ||
        rot_start < 0 || rot_start > D - rot_dim)
        return CSA2_ERR_SHAPE;
    if (x_tok_stride < 0 || out_tok_stride < 0 || x_head_stride < 0 || out_head_stride < 0 ||
        (H > 1 && (x_head_stride < D || out_head_stride < D)))
        return CSA2_ERR_SHAPE;
    // in place means the same element for the same channel
    if (x == out && ((T > 1 && x_tok_stride != out_tok_stride) ||
                     (H > 1 && x_head_stride != out_head_stride)))
        return CSA2_ERR_SHAPE;
    // no two rows of out may share an element: tokens outside heads or heads
    // outside tokens
    const int64_t tok_span = T > 1 ? (T - 1) * out_tok_stride + D : D;
    const int64_t head_span = (H - 1) * (H > 1 ? out_head_stride : 0) + D;
    if (T > 1 && (out_tok_stride < D ||
                  (H > 1 && out_tok_stride < head_span && out_head_stride < tok_span)))
        return CSA2_ERR_SHAPE;
    if (!aligned(x, dtype == CSA2_F32 ? 4 : 2) || !aligned(out, dtype == CSA2_F32 ? 4 : 2))
        return CSA2_ERR_ALIGN;
    if (T == 0) return CSA2_OK;
    rope::Args a{};
    a.x = x;
    a.out = out;
    a.pos = pos;
    a.freq = inv_freq;
    a.T = T;
    a.H = H;
    a.D = D;
    a.start = rot_start;
    a.rot = rot_dim;
    a.sign = inverse ? -1.0f : 1.0f;
    a.gain = mscale;
    a.xt = x_tok_stride;
    a.xh = x_head_stride;
    a.ot = out_tok_stride;
    a.oh = out_head_stride;
    const bool half = layout == CSA2_ROPE_HALF;
    return dtype == CSA2_F32 ? rope::launch<float>(a, half, (cudaStream_t)stream)
                             : rope::launch<__nv_bfloat16>(a, half, (cudaStream_t)stream);
}

extern "C" int csa2_rope_freqs(int rot_dim, double theta, int scaling, double factor,
                               int64_t orig_ctx, double beta_fast, double beta_slow,
                               double *inv_freq, void *stream) {
    using namespace csa2;
    if (!inv_freq) return CSA2_ERR_NULL;
    if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2) return CSA2_ERR_SHAPE;
    if (scaling < CSA2_ROPE_PLAIN || scaling > CSA2_ROPE_YARN || !(theta > 1.0) || !(factor >= 1.0))
        return CSA2_ERR_RANGE;
    double lo = 0.0, hi = 0.0;
    if (scaling == CSA2_ROPE_YARN) {
        if (orig_ctx < 1 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow)) return CSA2_ERR_RANGE;
        const double two_pi = 6.283185307179586477;
        auto pair_of = [&](double turns) {
            return rot_dim * log((double)orig_ctx / (two_pi * turns)) / (2.0 * log(theta));
        };
        lo = fmax(0.0, floor(pair_of(beta_fast)));
        hi = fmin(rot_dim - 1.0, ceil(pair_of(beta_slow)));
    }
    const int pairs = rot_dim / 2;
    return launch_kernel(false, rope::freqs_kernel, dim3((unsigned)(pairs + 127) / 128), dim3(128), 0,
                         (cudaStream_t)stream, pairs, theta, scaling, factor, lo, hi, inv_freq);
}
