// Attention of one new token over a paged FP4 cache: the tensor-core kernel.
// paged_attn.cu and paged_attn_mx.cu instantiate it for the two scale formats.
//
//   S^T[key, head]  = K Q^T        M = 64 keys, N = heads, K = channels
//   O^T[chan, head] += V^T P^T     M = 128 channels, N = heads, K = 64 keys
// with K = V = the dequantized rows. Keys and channels lie on the MMAs' rows, the
// heads of a group (16, 32 or 64; more heads are several groups) on their columns.
// S has M = 64, which runs at half rate: with 128 keys only one tile would fit.
//
// Work: every sequence is cut into tiles of 64 visible keys; the tiles of all
// (sequence, head group) pairs form one list that is divided evenly over the
// CTAs (one per SM), so that one long sequence and many short ones both fill the
// card. A CTA walks its share with an online softmax and keeps O^T in tensor
// memory; a pair that lies within one CTA is finished there, otherwise each CTA
// leaves (m, l, O) of its part and the combine kernel joins them.
//
// Roles of the 19 warps:
//   0-7   softmax: thread = a key and a quarter of the heads; warps 0-3 the first
//         half of the heads, 4-7 the second. Also the epilogue.
//   8-15  loads: codes and scales of the next tile in registers while the current
//         one is dequantized to shared memory; the queries.
//   16    issues S, 17 issues P V: each waits, suspended, for its own barriers.
//   18    the scout: page table entries, rows, and what the coming tiles are.
// Shared memory holds a ring of tiles, each ceil(C / 128) units of 64 keys x 128
// channels (16 KB), read by S as K (K-major) and by O as V (MN-major) from the same
// bytes. A tile is handed over in steps of two units, both ways.
//
// Bound (8 sequences of 128K, 64 heads, 512 channels): 137 GFLOP, 84 us at the
// measured bf16 rate; 303 MB, 46 us. M = 64 and N = 64 leave the MMAs at half of
// that rate at best (an MMA of 64 x 64 x 16 takes 35 cycles, one of 128 x 64 x 16
// 50), and they share shared memory with 64 KB of dequantized rows per tile.
// Measured steps: one thread polling two barriers 585 us (128-key tiles, one in
// the ring), rows read whole lines at a time and a warp that stays together 280, two
// issuing warps and bulk copies 268, the scout, which takes the walk and the
// table out of the load warps, 238, loads past L1 229, one buffer of weights 223, a
// prologue of one 32-bit scan 218, a faster joining kernel 216 (205 in a replayed
// graph). 128-key tiles (M = 128 for S) leave room for one tile: 292. 16 load warps,
// at 72 registers, spill: 342.
//
// Softmax: out = sum 2^(x_j - r) v_j / sum 2^(x_j - r) for any reference r. r is
// the head's maximum of its first tile and moves only when a score exceeds it
// by 2^8, so almost every tile needs no reduction over keys: a thread checks its
// own scores, one vote decides. l is kept per thread and summed over the keys
// once per sequence.
//
// Types. E4M3 scales: e2m1 x e4m3 has at most 6 significant bits and is a
// multiple of 2^-10 below 2^12, so f16 holds it exactly. Queries are bf16 (8
// bits); scaled by a power of two per head that brings their largest element
// to [2^13, 2^14) they are exact in f16 down to 2^-31 of that element, below which
// they round at 2^-25 absolute (2^-38 of it). Weights are rounded to f16: 2^-11
// relative, an eighth of the output's own bf16 rounding; they are kept below
// 2^15 by an offset of 7 in the exponent, so that weights down to 2^-21 of the
// reference keep all bits and those below 2^-32 vanish. The sum of weights is taken
// before they are rounded (its logarithm is the lse). What the rounding leaves is
// 3e-5 to 1.6e-4 of the output (2-norm) beside 1.65e-3 for the output's own, and
// changes 2 to 8 % of the outputs' bf16 values. E8M0 scales exceed f16's range:
// rows and queries are bf16 (exact), and the weights are two bf16 parts (16 bits),
// which costs a second P V: 8 sequences of 128K take 306 us, with E4M3 scales 205.
#pragma once

#include "fp4_rows.cuh"
#include "paged.cuh"
#include "tcgen05.cuh"

#include <type_traits>

namespace csa2 {
namespace pa {

// n / d for 0 <= n < 2^31 by a product (Granlund and Montgomery, "Division by
// Invariant Integers using Multiplication"): m = 2^(31 + s) / d rounded up with
// 2^s >= d is exact for such n, and below 2^32.
struct FastDiv {
    uint32_t m, s;
    __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
};
inline FastDiv fast_div(int d) {
    FastDiv f{0, 0};
    while ((1ll << f.s) < d) f.s++;
    f.m = (uint32_t)(((1ull << (31 + f.s)) + (uint64_t)d - 1) / (uint64_t)d);
    return f;
}

struct Args {
    const uint16_t *q;
    const uint8_t *fp4, *sf;
    PagedKv pk;
    const int64_t *ctx_len;
    int win, sink;         // 0: every position
    int cap;               // max_pages * page_size
    FastDiv page_div;      // by page_size
    int B, Hq, C, groups;  // groups of NH heads
    float scale;
    uint16_t *out;
    float *lse;
    // workspace
    int *flags;        // [G] a CTA that gave up a wait
    int *prefix;       // [B + 1] tiles before sequence b
    float *part_ml;    // [2 G][NH][2]: reference - P_OFFSET, sum
    float *part_o;     // [2 G][NH][128 U]
};

constexpr int TK = 64;              // keys per tile
constexpr int CHUNK = TK * 128;     // 64 channels of a tile: rows of 128 bytes
constexpr int UNIT = 2 * CHUNK;
constexpr int NSOFT = 256, NLOAD = 256, THREADS = NSOFT + NLOAD + 96;
constexpr int LOAD_WARPS = NLOAD / 32;
constexpr int S_WARP = (NSOFT + NLOAD) / 32, PV_WARP = S_WARP + 1, SCOUT_WARP = S_WARP + 2;
constexpr int ROW_RING = 4;          // tiles whose rows the scout has found ahead
constexpr int MAX_RING = 8;          // tiles of the ring, and steps
constexpr int VALID_RING = 16, QF_RING = 3;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float RESCALE_LOG2 = 8.0f;  // how far a score may exceed the reference
constexpr float P_OFFSET = 7.0f;      // weights are 2^(x - r + 7) <= 2^15
constexpr float REF_NONE = -3.0e38f;  // no key yet
constexpr uint64_t WAIT_NS = 200ull * 1000 * 1000;

// Visible keys of a sequence of n tokens: positions [0, ns) and [w0, n), listed
// in that order.
struct Seq {
    int nvis, ns, w0, tiles;
};
__device__ __forceinline__ Seq seq_of(const Args &a, int b) {
    const int64_t len = __ldg(a.ctx_len + b);
    const int n = len > a.cap ? a.cap : len < 0 ? 0 : (int)len;
    Seq s;
    s.ns = s.w0 = 0;
    if (a.win > 0) {
        s.ns = a.sink < n ? a.sink : n;
        s.w0 = n - a.win > s.ns ? n - a.win : s.ns;
    }
    s.nvis = s.ns + n - s.w0;
    s.tiles = (int)(((uint32_t)s.nvis + TK - 1) / TK);
    return s;
}

// T tiles are shared by min(G, T) CTAs, so that none between two that have tiles
// has none. Share c starts at c T / ctas: the larger shares lie apart (with all of
// them first, a batch that begins with short sequences took 5 % longer).
struct Shares {
    int T, ctas, each, more;
    __device__ __forceinline__ Shares(int T, int G) : T(T) {
        ctas = T < G ? T : G;
        each = ctas ? T / ctas : 0;
        more = T - each * ctas;
    }
    __device__ __forceinline__ int begin(int c) const { return c * each + c * more / ctas; }
    // the share with tile t: the last that starts at or before it
    __device__ __forceinline__ int owner(int t) const { return (int)((((int64_t)t + 1) * ctas - 1) / T); }
};

template <bool MX, int U, int NH>
struct Layout {
    static constexpr int PARTS = MX ? 2 : 1;       // of the weights
    static constexpr int NP = U == 4 && NH == 64 ? 1 : 2;  // buffers of weights (8 x 128K: 221 us with one, 233 with two)
    static constexpr int P_PART = TK * NH * 2;
    static constexpr int Q_CHUNK = NH * 128;       // 64 channels of Q
    static constexpr int Q_OFF = 0;
    static constexpr int P_OFF = Q_OFF + 2 * U * Q_CHUNK;
    static constexpr int K_OFF = P_OFF + NP * PARTS * P_PART;
    static constexpr int SMALL = 5120;
    static constexpr int FIT = (227 * 1024 - SMALL - K_OFF) / (U * UNIT);
    static constexpr int NS = (U + 1) / 2;                 // steps of a tile: two units each, the last maybe one
    static constexpr int NT = FIT * NS < MAX_RING ? FIT : MAX_RING / NS;  // tiles of the ring
    static_assert(NT >= 2, "two tiles fit the ring: P V of one beside S of the next");
    static constexpr int QF_OFF = K_OFF + NT * U * UNIT;      // fp32 [QF_RING][NH]
    static constexpr int REF_OFF = QF_OFF + QF_RING * NH * 4;   // fp32 [NH]: P_OFFSET - reference
    static constexpr int FAC_OFF = REF_OFF + NH * 4;      // fp32 [NH]: rescale factors, then 1 / l
    static constexpr int RED_OFF = FAC_OFF + NH * 4;      // fp32 [8][32]
    static constexpr int VALID_OFF = RED_OFF + 1024;      // a bit per key, 64 bits [VALID_RING]
    static constexpr int INFO_OFF = VALID_OFF + VALID_RING * 8;  // int4 [VALID_RING]
    static constexpr int ROW_OFF = INFO_OFF + VALID_RING * 16;    // int64 [ROW_RING][TK]: rows of the pool, -1: no key
    static constexpr int BAR_OFF = ROW_OFF + ROW_RING * TK * 8;
    static constexpr int B_QFULL = 0, B_QFREE = 1, B_UFULL = 2, B_UFREE = B_UFULL + MAX_RING,
                         B_SFULL = B_UFREE + MAX_RING, B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2,
                         B_PFREE = B_PFULL + 2, B_OFULL = B_PFREE + 2, B_OFREE = B_OFULL + 1,
                         B_RFULL = B_OFREE + 1, B_RFREE = B_RFULL + ROW_RING, NBARS = B_RFREE + ROW_RING;
    static constexpr int START_OFF = BAR_OFF + NBARS * 8; // int [3]: where the share starts
    static constexpr int TADDR_OFF = START_OFF + 24;
    static constexpr int ABORT_OFF = TADDR_OFF + 4;
    static constexpr int BYTES = ABORT_OFF + 4;
    static_assert(BYTES <= 227 * 1024, "shared memory budget");
    // TMEM: O^T unit u at columns u NH; S at U NH, a 64-row result fills 16 lanes of
    // each quadrant, buffer i those from 16 i on
    static constexpr uint32_t COLS_USED = (U + 1) * NH;
    static constexpr uint32_t COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static_assert(COLS_USED <= 512, "tensor memory");
};

static __device__ int g_paged_attn_error = 0;

static __device__ __forceinline__ void raise_abort(volatile int *abort) {
    *abort = 1;
    atomicExch(&g_paged_attn_error, 1);
}
// Wait for a phase, suspended in try_wait; false at once when the CTA has
// aborted, or, raising the abort, when WAIT_NS pass. Lanes may then differ: what
// holds warp-wide operations goes by all_ok of the lanes' answers.
static __device__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort) {
    if (test_wait(bar, parity)) return true;
    uint64_t t0 = 0;
    for (uint32_t it = 0;; it++) {
        if (try_wait(bar, parity)) return true;
        if (*abort) return false;
        if ((it & 63) == 63) {  // reading the timer takes as long as a short wait
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) {
                t0 = now;
            } else if (now - t0 > WAIT_NS) {
                raise_abort(abort);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool all_ok(bool ok) { return __all_sync(0xffffffffu, ok) != 0; }

// ---------------------------------------------------------------- tensor memory
// N columns (8, 16 or 32) of a warp's 32 lanes, thread t its lane t.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t ta, float (&v)[N]) {
    if constexpr (N == 32) {
        tmem_ld_32x32b_32(ta, v);
    } else if constexpr (N == 16) {
        tmem_ld_32x32b_16(ta, v);
    } else {
        static_assert(N == 8, "columns");
        uint32_t r[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(ta)
                     : "memory");
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                     :
                     : "memory");
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = __uint_as_float(r[i]);
    }
}
// N columns (4, 8 or 16) of 16 lanes: threads 0-15 read columns [0, N), threads
// 16-31 columns [N, 2 N).
template <int N>
__device__ __forceinline__ void tmem_load_half(uint32_t ta, float (&v)[N]) {
    uint32_t r[N];
    if constexpr (N == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
            "%12, %13, %14, %15}, [%16], 16;"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(ta));
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8], 8;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(ta));
    } else {
        static_assert(N == 4, "columns");
        asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x4.b32 {%0, %1, %2, %3}, [%4], 4;"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(ta));
    }
#pragma unroll
    for (int i = 0; i < N; i += 4)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])
                     :
                     : "memory");
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t ta, const float (&v)[N]) {
    if constexpr (N == 32) {
        tmem_st_32x32b_32(ta, v);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(ta + i),
                         "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1])), "r"(__float_as_uint(v[i + 2])),
                         "r"(__float_as_uint(v[i + 3])), "r"(__float_as_uint(v[i + 4])),
                         "r"(__float_as_uint(v[i + 5])), "r"(__float_as_uint(v[i + 6])),
                         "r"(__float_as_uint(v[i + 7]))
                         : "memory");
    }
}

// Sums of N <= 16 values over each half of the warp: lane i (mod N) of a half
// receives that of value i.
template <int N>
__device__ __forceinline__ float columns_sum(float (&x)[N], int lane) {
#pragma unroll
    for (int w = N / 2; w >= 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; i++) {
            const float send = up ? x[i] : x[i + w], keep = up ? x[i + w] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, w);
        }
    }
#pragma unroll
    for (int b = N; b < 16; b <<= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], b);
    return x[0];
}
// The same for the maximum; NaN counts as -inf.
template <int N>
__device__ __forceinline__ float columns_max(float (&x)[N], int lane) {
#pragma unroll
    for (int w = N / 2; w >= 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; i++) {
            const float send = up ? x[i] : x[i + w], keep = up ? x[i + w] : x[i];
            x[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, w));
        }
    }
#pragma unroll
    for (int b = N; b < 16; b <<= 1) x[0] = fmaxf(x[0], __shfl_xor_sync(0xffffffffu, x[0], b));
    return x[0] == x[0] ? x[0] : -INFINITY;
}

// True in one lane of a warp that is together, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Where a CTA stands in the list of tiles.
struct Walk {
    int b, g;        // sequence and head group
    int tile;        // of the sequence
    Seq s;
    // to the next tile; the caller never walks past its last
    __device__ __forceinline__ void next(const Args &a, bool more) {
        if (++tile < s.tiles || !more) return;
        tile = 0;
        if (++g < a.groups) return;
        g = 0;
        do {
            s = seq_of(a, ++b);
        } while (s.tiles == 0);
    }
    // position of key r of this tile, -1 if there is none
    __device__ __forceinline__ int position(int r) const {
        const int64_t j = (int64_t)tile * TK + r;
        return j >= s.nvis ? -1 : (int)(j < s.ns ? j : s.w0 + j - s.ns);
    }
    // keys of this tile, rounded up to the 16 of an MMA step
    __device__ __forceinline__ int keys16() const {
        const int k = s.nvis - tile * TK;
        return k >= TK ? TK : (k + 15) & ~15;
    }
};

// Byte offset of 16-byte piece p of key row k in a tile of weights with rows of
// 2 NH bytes, in the swizzle of that width.
template <int NH>
__device__ __forceinline__ uint32_t p_offset(int k, int p) {
    if constexpr (NH == 64) return sw128(k, p);
    if constexpr (NH == 32) return (uint32_t)(k * 64 + ((p ^ ((k >> 1) & 3)) << 4));
    return (uint32_t)(k * 32 + ((p ^ ((k >> 2) & 1)) << 4));
}
template <int NH>
__device__ __forceinline__ uint64_t p_desc(uint32_t addr) {
    if constexpr (NH == 64) return sdesc_sw<2>(addr, 16, 1024);
    if constexpr (NH == 32) return sdesc_sw<4>(addr, 16, 512);
    return sdesc_sw<6>(addr, 16, 256);
}

// What the scout tells the other roles about a tile, beside its keys.
struct TileInfo {
    int b, g;   // sequence and head group
    int flags;  // kLast, kWhole, and the 16-key steps of P V
    int slot;   // where this CTA's part of the pair goes
};
constexpr int kLast = 1;   // the CTA's last tile of the pair
constexpr int kWhole = 2;  // the CTA has all tiles of the pair
constexpr int kFirst = 4;  // the CTA's first tile of the pair
__device__ __forceinline__ TileInfo read_info(uint32_t info, uint32_t i) {
    TileInfo v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.b), "=r"(v.g), "=r"(v.flags), "=r"(v.slot)
                 : "r"(info + 16 * i)
                 : "memory");
    return v;
}

// A position in a ring of N and the parity of its round.
template <int N>
struct Ring {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

template <bool MX, int U, int NH>
__global__ void __launch_bounds__(THREADS, 1) attn_kernel(const Args a) {
    using L = Layout<MX, U, NH>;
    constexpr int NG = NH / 2;            // heads of a group of four softmax warps
    constexpr int NC = NH / 4;            // heads per softmax thread
    constexpr int W = NG < 16 ? NG : 16;  // columns of O^T in registers at a time
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t base = smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int *abort = reinterpret_cast<volatile int *>(sm + L::ABORT_OFF);
    auto bar = [&](uint32_t i) { return base + L::BAR_OFF + 8u * i; };
    const int G = gridDim.x, cta = blockIdx.x;

    if (tid == 0) {
        mbar_init(bar(L::B_QFULL), LOAD_WARPS);
        mbar_init(bar(L::B_QFREE), 1);
        for (int i = 0; i < L::NT * L::NS; i++) {
            mbar_init(bar(L::B_UFULL + i), LOAD_WARPS);  // step s of ring tile t: t NS + s
            mbar_init(bar(L::B_UFREE + i), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(bar(L::B_SFULL + i), 1);
            mbar_init(bar(L::B_SFREE + i), NSOFT / 32);
            mbar_init(bar(L::B_PFULL + i), NSOFT / 32);
            mbar_init(bar(L::B_PFREE + i), 1);
        }
        mbar_init(bar(L::B_OFULL), 1);
        mbar_init(bar(L::B_OFREE), NSOFT / 32);
        for (int i = 0; i < ROW_RING; i++) {
            mbar_init(bar(L::B_RFULL + i), 1);
            mbar_init(bar(L::B_RFREE + i), LOAD_WARPS);
        }
        *abort = (base & 1023u) != 0;  // the swizzles want this alignment
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == S_WARP) tmem_alloc(base + L::TADDR_OFF, L::COLS);

    grid_dep_wait();
    grid_dep_launch();
    // ---- this CTA's share of the tiles: the prefix of the sequences' tiles, chunk by
    // chunk of THREADS of them; one chunk, and one pass, for any usual batch
    int *red = reinterpret_cast<int *>(sm + L::RED_OFF);
    int *start = reinterpret_cast<int *>(sm + L::START_OFF);  // tile of the pair, b, g
    constexpr int WARPS = THREADS / 32;
    static_assert(WARPS <= 32, "a warp scans the warps' sums");
    // tiles before this thread's sequence of a chunk; `sum` receives the chunk's
    auto scan = [&](int v, int &sum) {
        int x = v;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        __syncthreads();
        if (lane == 31) red[warp] = x;
        __syncthreads();
        int s = lane < WARPS ? red[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        sum = __shfl_sync(0xffffffffu, s, 31);
        const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
        return (warp > 0 ? before : 0) + x - v;
    };
    auto tiles_of = [&](int b) { return b < a.B ? seq_of(a, b).tiles : 0; };
    int v = tiles_of(tid), sum, at = scan(v, sum), total = sum;
    for (int b0 = THREADS; b0 < a.B; b0 += THREADS) {
        int more;
        scan(tiles_of(b0 + tid), more);
        total += more;
    }
    const Shares shares(total * a.groups, G);
    const int t_begin = cta < shares.ctas ? shares.begin(cta) : 0;
    const int n_tiles = cta < shares.ctas ? shares.begin(cta + 1) - t_begin : 0;
    for (int b0 = 0, before = 0; b0 < a.B; b0 += THREADS) {
        if (b0 > 0) {
            before += sum;
            v = tiles_of(b0 + tid);
            at = scan(v, sum);
        }
        const int b = b0 + tid, first = (before + at) * a.groups;
        if (cta == 0 && b < a.B) a.prefix[b] = before + at;
        if (n_tiles > 0 && first <= t_begin && t_begin < first + v * a.groups) {
            start[2] = (t_begin - first) / v;
            start[0] = t_begin - first - start[2] * v;
            start[1] = b;
        }
    }
    if (cta == 0 && tid == 0) a.prefix[a.B] = total;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sm + L::TADDR_OFF);
    Walk w{};
    if (n_tiles > 0) {
        w.tile = start[0];
        w.b = start[1];
        w.g = start[2];
        w.s = seq_of(a, w.b);
    }

    if (n_tiles == 0 || *abort) {
        // nothing to do
    } else if (warp < NSOFT / 32) {
        // ------------------------------------------------ softmax and epilogue
        const int quad = warp & 3, part = warp >> 2;  // lanes of TMEM, half of the heads
        const int key = quad * 16 + (lane & 15), hq = lane >> 4;  // a thread: a key, a quarter of the heads
        const int gt = tid & 127;
        const int bar_id = 1 + part;
        const uint32_t lanes = (uint32_t)(32 * quad) << 16;
        // of this half of the heads
        float *ref = reinterpret_cast<float *>(sm + L::REF_OFF) + part * NG;
        float *fac = reinterpret_cast<float *>(sm + L::FAC_OFF) + part * NG;
        float *red_f = reinterpret_cast<float *>(sm + L::RED_OFF) + part * 128;  // [4][NG]
        const volatile uint16_t *valid = reinterpret_cast<const volatile uint16_t *>(sm + L::VALID_OFF);
        bool ok = true, first = true;
        float l[NC];
        uint32_t seg = 0;
        Ring<2> sr;
        Ring<L::NP> pr;
        Ring<L::NT> ur;
        for (int k = 0; k < n_tiles; k++) {
            if (first) {
#pragma unroll
                for (int i = 0; i < NC; i++) l[i] = 0.0f;
            }
            const float *qf = reinterpret_cast<const float *>(sm + L::QF_OFF) + (seg % QF_RING) * NH + part * NG + hq * NC;
            const float *rq = ref + hq * NC;
            // the step's barrier carries on what the scout wrote before the load warps'
            // arrival (valid, info), and the load warps' qf
            ok = wait_bar(bar(L::B_UFULL + ur.i * L::NS), ur.phase, abort) && ok;
            const uint32_t vi = (uint32_t)k % VALID_RING;
            const TileInfo info = read_info(base + L::INFO_OFF, vi);
            const uint32_t seen = ok ? valid[vi * 4 + quad] : 0u;
            const bool see = (seen >> (lane & 15)) & 1;
            ok = wait_bar(bar(L::B_SFULL + sr.i), sr.phase, abort) && ok;
            tc_fence_after();
            // x becomes the exponents x f + (7 - reference)
            float x[NC];
            auto exponents = [&]() {
                tmem_load_half<NC>(tmem + lanes + ((16u * sr.i) << 16) + U * NH + part * NG, x);
#pragma unroll
                for (int i = 0; i < NC; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(qf + i);
                    const float4 r = *reinterpret_cast<const float4 *>(rq + i);
                    x[i] = fmaf(x[i], f.x, r.x);
                    x[i + 1] = fmaf(x[i + 1], f.y, r.y);
                    x[i + 2] = fmaf(x[i + 2], f.z, r.z);
                    x[i + 3] = fmaf(x[i + 3], f.w, r.w);
                }
            };
            // ---- does a score exceed its head's reference by 2^8? The vote also tells of a
            // wait that ran out; the group then leaves the loop together, so that its
            // barriers never part.
            bool move = first;
            if (!first) {
                exponents();
                float over = x[0];
#pragma unroll
                for (int i = 1; i < NC; i++) over = fmaxf(over, x[i]);
                move = named_bar_or(bar_id, 128, !ok || (see && over > RESCALE_LOG2 + P_OFFSET));
            }
            if (move) {
                if (named_bar_or(bar_id, 128, !ok)) break;
                // rare: the scores are read again
                float y[NC];
                tmem_load_half<NC>(tmem + lanes + ((16u * sr.i) << 16) + U * NH + part * NG, y);
#pragma unroll
                for (int i = 0; i < NC; i++) y[i] = see ? y[i] * qf[i] : -INFINITY;
                const float mine = columns_max<NC>(y, lane);
                if ((lane & 15) < NC) red_f[quad * NG + hq * NC + (lane & 15)] = mine;
                named_bar_sync(bar_id, 128);
                if (gt < NG) {
                    const float m = fmaxf(fmaxf(red_f[gt], red_f[NG + gt]), fmaxf(red_f[2 * NG + gt], red_f[3 * NG + gt]));
                    const float old = P_OFFSET - ref[gt];
                    const bool up = first || m > old + RESCALE_LOG2;
                    const float now = up ? fmaxf(m, REF_NONE) : old;
                    fac[gt] = first || !up ? 1.0f : ex2(old - now);
                    if (up) ref[gt] = P_OFFSET - now;
                }
                named_bar_sync(bar_id, 128);
            }
            // this buffer's last P V is done, and with one buffer so is the last
            // tile's; with two, a rescale waits for the other one too
            ok = wait_bar(bar(L::B_PFREE + pr.i), pr.phase ^ 1, abort) && ok;
            if (move) exponents();  // with the new references
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::B_SFREE + sr.i));
            if (move && !first) {
                if constexpr (L::NP == 2)
                    ok = wait_bar(bar(L::B_PFREE + (pr.i ^ 1)), pr.i ? pr.phase : pr.phase ^ 1, abort) && ok;
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < U; u++)
#pragma unroll 1
                    for (int c = 0; c < NG; c += W) {
                        const uint32_t ta = tmem + lanes + u * NH + part * NG + c;
                        float o[W];
                        tmem_load<W>(ta, o);
#pragma unroll
                        for (int i = 0; i < W; i++) o[i] *= fac[c + i];
                        tmem_store<W>(ta, o);
                    }
                tmem_st_wait();
#pragma unroll
                for (int i = 0; i < NC; i++) l[i] *= fac[hq * NC + i];
            }
            const uint32_t pb = base + L::P_OFF + pr.i * L::PARTS * L::P_PART;
#pragma unroll
            for (int i = 0; i < NC; i++) x[i] = ex2(x[i]);
            if (!see) {  // a row without a key may hold anything
#pragma unroll
                for (int i = 0; i < NC; i++) x[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < NC; i++) l[i] += x[i];
            uint32_t v[NC / 2], v2[NC / 2];  // weights, and (MX) what their rounding leaves
#pragma unroll
            for (int i = 0; i < NC / 2; i++) {
                if constexpr (MX) {
                    v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                    v2[i] = pack_bf16x2(x[2 * i] - bf16_lo(v[i]), x[2 * i + 1] - bf16_hi(v[i]));
                } else {
                    v[i] = pack_f16x2(x[2 * i], x[2 * i + 1]);
                }
            }
            // the thread's heads of its key's row: 2 NC bytes
            const int byte0 = (part * NG + hq * NC) * 2;
            if constexpr (NC >= 8) {
#pragma unroll
                for (int p = 0; p < NC / 8; p++) {
                    const uint32_t off = p_offset<NH>(key, byte0 / 16 + p);
                    st_shared_v4(pb + off, make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]));
                    if constexpr (MX)
                        st_shared_v4(pb + L::P_PART + off,
                                     make_uint4(v2[4 * p], v2[4 * p + 1], v2[4 * p + 2], v2[4 * p + 3]));
                }
            } else {
                const uint32_t off = p_offset<NH>(key, byte0 / 16) + byte0 % 16;
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(pb + off), "r"(v[0]), "r"(v[1]) : "memory");
                if constexpr (MX)
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(pb + L::P_PART + off), "r"(v2[0]), "r"(v2[1])
                                 : "memory");
            }
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::B_PFULL + pr.i));
            sr.next();
            pr.next();
            ur.next();

            first = info.flags & kLast;
            if (first) {
                // ---- the pair's part of this CTA is done
                const bool whole = info.flags & kWhole;
                const float s = columns_sum<NC>(l, lane);
                if ((lane & 15) < NC) red_f[quad * NG + hq * NC + (lane & 15)] = s;
                named_bar_sync(bar_id, 128);
                const int h0 = info.g * NH + part * NG;
                if (gt < NG) {
                    const float sum = red_f[gt] + red_f[NG + gt] + red_f[2 * NG + gt] + red_f[3 * NG + gt];
                    fac[gt] = sum != 0.0f ? 1.0f / sum : 0.0f;
                    if (!whole) {
                        float *ml = a.part_ml + ((int64_t)info.slot * NH + part * NG + gt) * 2;
                        ml[0] = -ref[gt];
                        ml[1] = sum;
                    } else if (a.lse && h0 + gt < a.Hq) {
                        a.lse[(int64_t)info.b * a.Hq + h0 + gt] =
                            sum != 0.0f ? (log2f(sum) - ref[gt]) * LN2 : -INFINITY;
                    }
                }
                named_bar_sync(bar_id, 128);
                ok = wait_bar(bar(L::B_OFULL), seg & 1, abort) && ok;
                tc_fence_after();
#pragma unroll 1
                for (int u = 0; u < U; u++) {
                    const int ch = 128 * u + quad * 32 + lane;
#pragma unroll 1
                    for (int c = 0; c < NG; c += W) {
                        float o[W];
                        tmem_load<W>(tmem + lanes + u * NH + part * NG + c, o);
                        if (ch >= a.C) continue;
                        if (whole) {
                            uint16_t *dst = a.out + ((int64_t)info.b * a.Hq + h0 + c) * a.C + ch;
#pragma unroll
                            for (int i = 0; i < W; i++)
                                if (h0 + c + i < a.Hq) {
                                    const __nv_bfloat16 v = __float2bfloat16_rn(o[i] * fac[c + i]);
                                    dst[(int64_t)i * a.C] = *reinterpret_cast<const uint16_t *>(&v);
                                }
                        } else {
                            float *dst = a.part_o + ((int64_t)info.slot * NH + part * NG + c) * (128 * U) + ch;
#pragma unroll
                            for (int i = 0; i < W; i++) dst[i * (128 * U)] = o[i];
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_OFREE));
                seg++;
            }
        }
    } else if (warp < S_WARP) {
        // ------------------------------------------------ loads and dequantization
        // A warp has eight rows of the tile, two per thread. Per step a row is 128 bytes of codes, eight
        // lanes of 16 bytes: four whole lines per access (with a lane per row an access
        // touched 32, and the load pipe held up everything else). The lanes' order
        // gives each eight of a store's lanes four rows and two pieces: all banks.
        const int lw = warp - NSOFT / 32;
        const int piece = (lane & 1) | (lane >> 3) << 1;      // 32 channels of a step
        const int r = lw * 8 + ((lane >> 1) & 3);             // key rows r and r + 4
        // in a step: row r, and the swizzled place of its piece i: swap ^ (i << 4); row
        // r + 4 lies 512 bytes on, and 64 swapped
        const uint32_t row_off = (piece >> 1) * CHUNK + (r >> 3) * 1024 + (r & 7) * 128;
        const uint32_t swap = (uint32_t)(((piece & 1) * 4) ^ (r & 7)) << 4;
        const int row_bytes = a.C / 2, sf_bytes = a.C / (MX ? 32 : 16);
        bool ok = true;
        uint32_t seg = 0;
        Ring<L::NT> ur;
        Ring<ROW_RING> rr;
        uint4 code[L::NS][2];
        uint32_t scl[L::NS][2];  // one E8M0 byte, or two E4M3; as loaded
        auto load_tile = [&]() {
            ok = all_ok(wait_bar(bar(L::B_RFULL + rr.i), rr.phase, abort) && ok);
            const volatile int64_t *rows = reinterpret_cast<const volatile int64_t *>(sm + L::ROW_OFF) + rr.i * TK + r;
            const int64_t row[2] = {rows[0], rows[4]};
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::B_RFREE + rr.i));
            rr.next();
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const uint8_t *c = a.fp4 + row[j] * row_bytes + 16 * piece;
                const uint8_t *s = a.sf + row[j] * sf_bytes + (MX ? piece : 2 * piece);
#pragma unroll
                for (int st = 0; st < L::NS; st++) {
                    code[st][j] = make_uint4(0, 0, 0, 0);
                    scl[st][j] = 0;
                    if (ok && row[j] >= 0 && 256 * st + 32 * piece < a.C) {
                        code[st][j] = ld_stream_v4(c + 128 * st);
                        scl[st][j] = MX ? (uint32_t)__ldg(s + 8 * st)
                                        : (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(s + 16 * st));
                    }
                }
            }
        };
        load_tile();
        for (int k = 0; k < n_tiles; k++) {
            const TileInfo info = read_info(base + L::INFO_OFF, (uint32_t)k % VALID_RING);
            const int keys = (info.flags >> 8) * 16;
            if (ok && (info.flags & kFirst)) {
                // ---- queries of a new pair: one warp a head, lanes over channels
                ok = wait_bar(bar(L::B_QFREE), (seg & 1) ^ 1, abort) && ok;
                float *qf = reinterpret_cast<float *>(sm + L::QF_OFF) + (seg % QF_RING) * NH;
                constexpr int MINE = NH / LOAD_WARPS, HB = U > 2 || MINE < 4 ? 2 : 4;  // heads of a warp, and at a time
#pragma unroll 1
                for (int h0 = 0; h0 < MINE; h0 += HB) {
                    uint4 v[HB][(U + 1) / 2];  // all loads before the first use
#pragma unroll
                    for (int j = 0; j < HB; j++) {
                        const int h = info.g * NH + (h0 + j) * LOAD_WARPS + lw;
                        const uint16_t *q = a.q + ((int64_t)info.b * a.Hq + h) * a.C;
#pragma unroll
                        for (int i = 0; i < (U + 1) / 2; i++) {
                            const int c = 256 * i + 8 * lane;
                            v[j][i] = make_uint4(0, 0, 0, 0);
                            if (h < a.Hq && c < a.C) v[j][i] = __ldg(reinterpret_cast<const uint4 *>(q + c));
                        }
                    }
#pragma unroll
                    for (int j = 0; j < HB; j++) {
                        const int h = (h0 + j) * LOAD_WARPS + lw;
                        float mul = 1.0f, f = a.scale * LOG2E;
                        if constexpr (!MX) {
                            uint32_t top = 0;  // largest |q| as bf16 bits (NaN and inf above all others)
#pragma unroll
                            for (int i = 0; i < (U + 1) / 2; i++) {
                                const uint32_t u4[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
#pragma unroll
                                for (int e = 0; e < 4; e++) top = max(top, max(u4[e] & 0x7FFF, (u4[e] >> 16) & 0x7FFF));
                            }
                            top = __reduce_max_sync(0xffffffffu, top);
                            // 2^e with the top exponent brought to 13; e <= 100 keeps 2^e in range
                            int e = 13 - ((int)(top >> 7) - 127);
                            e = e > 100 ? 100 : e;
                            mul = __uint_as_float((uint32_t)(e + 127) << 23);
                            f *= __uint_as_float((uint32_t)(127 - e) << 23);
                        }
                        if (lane == 0) qf[h] = f;
#pragma unroll
                        for (int i = 0; i < (U + 1) / 2; i++) {
                            const int c = 256 * i + 8 * lane;
                            if (c >= 128 * U) continue;
                            uint32_t u4[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
                            if constexpr (!MX) {
#pragma unroll
                                for (int e = 0; e < 4; e++)
                                    u4[e] = pack_f16x2(bf16_lo(u4[e]) * mul, bf16_hi(u4[e]) * mul);
                            }
                            st_shared_v4(base + L::Q_OFF + (c >> 6) * L::Q_CHUNK + sw128(h, (c >> 3) & 7),
                                         make_uint4(u4[0], u4[1], u4[2], u4[3]));
                        }
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_QFULL));
                seg++;
            }
#pragma unroll
            for (int st = 0; st < L::NS; st++) {
                ok = wait_bar(bar(L::B_UFREE + ur.i * L::NS + st), ur.phase ^ 1, abort) && ok;
                if (8 * lw < keys && 256 * st + 32 * piece < a.C) {
                    const uint32_t dst = base + L::K_OFF + (ur.i * U + 2 * st) * UNIT + row_off;
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const uint32_t wd[4] = {code[st][j].x, code[st][j].y, code[st][j].z, code[st][j].w};
                        if constexpr (MX) {
                            const MxScale s = mx_scale(scl[st][j]);
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                st_shared_v4(dst + 512 * j + (swap ^ ((i + 4 * j) << 4)), rows_bf16(wd[i], s));
                        } else {
                            uint32_t s01;  // the two groups' scales in f16
                            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s01) : "h"((uint16_t)scl[st][j]));
                            const uint32_t s[2] = {__byte_perm(s01, 0, 0x1010), __byte_perm(s01, 0, 0x3232)};
#pragma unroll
                            for (int i = 0; i < 4; i++)
                                st_shared_v4(dst + 512 * j + (swap ^ ((i + 4 * j) << 4)), rows_f16(wd[i], s[i >> 1]));
                        }
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_UFULL + ur.i * L::NS + st));
            }
            ur.next();
            // after this tile's last fence, which would wait for them
            if (k + 1 < n_tiles) load_tile();
        }
    } else if (warp == SCOUT_WARP) {
        // ------------------------------------------------ the scout: where the rows of the
        // coming tiles lie, which keys there are, and what the tile is. Table entries are
        // looked at one tile after they were asked for.
        bool ok = true;
        Ring<ROW_RING> rr;
        Walk ahead = w;
        int32_t page[2];
        int slot[2];
        auto look_up = [&]() {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int pos = ahead.position(lane + 32 * j);
                const int e = pos < 0 ? 0 : a.page_div(pos);
                slot[j] = pos - e * a.pk.page_size;
                page[j] = pos < 0 ? -1 : __ldg(a.pk.table + (int64_t)ahead.b * a.pk.max_pages + e);
            }
        };
        look_up();
        for (int k = 0; k < n_tiles && all_ok(ok); k++) {
            int64_t row[2];
#pragma unroll
            for (int j = 0; j < 2; j++)
                row[j] = page[j] >= 0 && page[j] < a.pk.n_pages ? (int64_t)page[j] * a.pk.page_size + slot[j] : -1;
            if (k + 1 < n_tiles) {
                ahead.next(a, true);
                look_up();
            }
            const uint32_t lo = __ballot_sync(0xffffffffu, row[0] >= 0), hi = __ballot_sync(0xffffffffu, row[1] >= 0);
            ok = wait_bar(bar(L::B_RFREE + rr.i), rr.phase ^ 1, abort) && ok;
            volatile int64_t *to = reinterpret_cast<volatile int64_t *>(sm + L::ROW_OFF) + rr.i * TK;
            to[lane] = row[0];
            to[lane + 32] = row[1];
            if (lane == 0) {
                const uint32_t vi = (uint32_t)k % VALID_RING;
                volatile uint32_t *v = reinterpret_cast<volatile uint32_t *>(sm + L::VALID_OFF) + 2 * vi;
                v[0] = lo;
                v[1] = hi;
                const bool end_seq = w.tile + 1 == w.s.tiles;
                const bool from_start = w.tile <= k;  // the pair's first tile is this CTA's too
                const int flags = (end_seq || k + 1 == n_tiles ? kLast : 0) | (end_seq && from_start ? kWhole : 0) |
                                  (k == 0 || w.tile == 0 ? kFirst : 0) | (w.keys16() / 16) << 8;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(base + L::INFO_OFF + 16 * vi), "r"(w.b),
                             "r"(w.g), "r"(flags), "r"(2 * cta + (w.tile < k ? 1 : 0))
                             : "memory");
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::B_RFULL + rr.i));
            rr.next();
            w.next(a, k + 1 < n_tiles);
        }
    } else if (warp == S_WARP) {
        // ------------------------------------------------ issue of S. The two issuing
        // warps each wait for their own barriers, suspended: one warp that watched both
        // kept the shared-memory pipe busy with its polls. A warp stays together, so that
        // descriptors are computed once for it, and one lane issues.
        constexpr uint32_t id = MX ? idesc_bf16(TK, NH, false) : idesc_f16(TK, NH, false);
        const uint64_t dq = sdesc(base + L::Q_OFF, 16, 1024);
        const uint64_t dk = sdesc(base + L::K_OFF, 16, 1024);
        bool ok = true, first = true;
        uint32_t seg = 0;
        Ring<2> sr;
        Ring<L::NT> ur;
        for (int k = 0; k < n_tiles && all_ok(ok); k++) {
            if (first) ok = wait_bar(bar(L::B_QFULL), seg & 1, abort) && ok;
            ok = wait_bar(bar(L::B_SFREE + sr.i), sr.phase ^ 1, abort) && ok;
            const uint32_t sd = tmem + ((16u * sr.i) << 16) + U * NH;
            bool last = false;
#pragma unroll 1
            for (int st = 0; st < L::NS; st++) {
                ok = wait_bar(bar(L::B_UFULL + ur.i * L::NS + st), ur.phase, abort) && ok;
                if (st == 0) last = read_info(base + L::INFO_OFF, (uint32_t)k % VALID_RING).flags & kLast;
                __syncwarp();
                tc_fence_after();
                const uint64_t k0 = dk + (uint64_t)(((ur.i * U + 2 * st) * UNIT) >> 4);
                const uint64_t q0 = dq + (uint64_t)((st * 4 * L::Q_CHUNK) >> 4);
                const int left = (a.C - 256 * st) / 16;  // 16-channel MMAs, eight a unit
                if (elect_one()) {
                    auto step = [&](int s, uint32_t acc) {
                        mma_bf16(sd, k0 + (uint64_t)(((s >> 2) * CHUNK + (s & 3) * 32) >> 4),
                                 q0 + (uint64_t)(((s >> 2) * L::Q_CHUNK + (s & 3) * 32) >> 4), id, acc);
                    };
                    step(0, st > 0 ? 1u : 0u);
                    if (left >= 16) {
#pragma unroll
                        for (int s = 1; s < 16; s++) step(s, 1u);
                    } else {
#pragma unroll 1
                        for (int s = 1; s < left; s++) step(s, 1u);
                    }
                    if (st == L::NS - 1) {
                        mma_commit(bar(L::B_SFULL + sr.i));
                        if (last) mma_commit(bar(L::B_QFREE));
                    }
                }
                __syncwarp();
            }
            ur.next();
            sr.next();
            first = last;
            seg += last;
        }
    } else {
        // ------------------------------------------------ issue of P V
        constexpr uint32_t id = MX ? idesc_bf16(128, NH, true, true) : idesc_f16(128, NH, true, true);
        const uint64_t dv = sdesc(base + L::K_OFF, CHUNK, 1024);
        const uint64_t dp = p_desc<NH>(base + L::P_OFF);
        bool ok = true, first = true;
        uint32_t seg = 0;
        Ring<L::NP> pr;
        Ring<L::NT> ur;
        for (int k = 0; k < n_tiles && all_ok(ok); k++) {
            // this barrier carries the scout's info on to here
            ok = wait_bar(bar(L::B_UFULL + ur.i * L::NS), ur.phase, abort) && ok;
            const int flags = read_info(base + L::INFO_OFF, (uint32_t)k % VALID_RING).flags, steps = flags >> 8;
            const bool last = flags & kLast;
            if (first) ok = wait_bar(bar(L::B_OFREE), (seg & 1) ^ 1, abort) && ok;
            ok = wait_bar(bar(L::B_PFULL + pr.i), pr.phase, abort) && ok;
            __syncwarp();
            tc_fence_after();
            const uint64_t p0 = dp + (uint64_t)((pr.i * L::PARTS * L::P_PART) >> 4);
            const uint64_t v0 = dv + (uint64_t)((ur.i * U * UNIT) >> 4);
            if (elect_one()) {
#pragma unroll
                for (int u = 0; u < U; u++) {
                    auto step = [&](int s, uint32_t acc) {
                        const uint64_t vd = v0 + (uint64_t)((u * UNIT + s * 2048) >> 4);
                        const uint64_t pd = p0 + (uint64_t)((s * 16 * NH * 2) >> 4);
                        mma_bf16(tmem + u * NH, vd, pd, id, acc);
                        if constexpr (MX) mma_bf16(tmem + u * NH, vd, pd + (uint64_t)(L::P_PART >> 4), id, 1u);
                    };
                    step(0, first ? 0u : 1u);
                    if (steps == TK / 16) {
#pragma unroll
                        for (int s = 1; s < TK / 16; s++) step(s, 1u);
                    } else {
#pragma unroll 1
                        for (int s = 1; s < steps; s++) step(s, 1u);
                    }
                    if (u % 2 || u == U - 1) mma_commit(bar(L::B_UFREE + ur.i * L::NS + u / 2));
                }
                mma_commit(bar(L::B_PFREE + pr.i));
                if (last) mma_commit(bar(L::B_OFULL));
            }
            __syncwarp();
            ur.next();
            pr.next();
            first = last;
            seg += last;
        }
    }
    __syncthreads();
    if (tid == 0) a.flags[cta] = *abort;
    if (*abort) {
        // MMAs still in flight land before the CTA's memory is released
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    if (warp == S_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, L::COLS);
    }
}

template <bool MX, int U, int NH>
int launch_one(const Args &a, int G, cudaStream_t s) {
    using L = Layout<MX, U, NH>;
    static PerDevice smem_set;
    if (!set_smem_limit_once(smem_set, attn_kernel<MX, U, NH>, L::BYTES)) return CSA2_ERR_CUDA;
    return launch_kernel(true, attn_kernel<MX, U, NH>, dim3((unsigned)G), dim3(THREADS), L::BYTES, s, a);
}

// The kernel for C channels and head groups of nh.
template <bool MX>
int launch_attn(const Args &a, int nh, int G, cudaStream_t s) {
    const int u = (a.C + 127) / 128;
#define CSA2_PA(U_)                                       \
    if (u == U_) {                                        \
        if (nh == 16) return launch_one<MX, U_, 16>(a, G, s); \
        if (nh == 32) return launch_one<MX, U_, 32>(a, G, s); \
        return launch_one<MX, U_, 64>(a, G, s);           \
    }
    CSA2_PA(1)
    CSA2_PA(2)
    CSA2_PA(3)
    CSA2_PA(4)
#undef CSA2_PA
    return CSA2_ERR_SHAPE;
}

int launch_paged_attn_fp4(const Args &a, int nh, int G, cudaStream_t s);
int launch_paged_attn_mxfp4(const Args &a, int nh, int G, cudaStream_t s);

}  // namespace pa
}  // namespace csa2
