// Page management of the paged FP4 cache: extend, fork, free, copy, compact.
//
// The free pages are listed once per call, ascending, by a prefix count over
// the reference counts (4096 pages per CTA; beyond one CTA's share a counting
// launch goes first). Requests take pages by their rank among the requests, so
// nothing depends on the order in which blocks run: the only atomics add to
// integers whose sum has no order.
//
// Tables and counts are a few MB at most and latency-bound; the page bodies are
// bound by memory, read once and written once. Free, fork and copy for 8 forks of 4K
// tokens take 8.0 us, for 256 forks of 32K (77 MB) 22.7; compaction of 8192 pages of
// which 60 % are in use (589 MB) 104.5 us, 5.6 TB/s. Extension walks every row from its
// start, by one warp to count and again where an entry is missing: 32 sequences of 4K in
// pages of 16 take 5.7 us with nothing missing and 6.8 with a page each; of 256K in
// pages of 64 8.0 and 16.3; of 1M 18.6 and 49.5, in pages of 16 62 and 294.
#include "paged.cuh"

#include <type_traits>

namespace csa2 {
namespace pages {

constexpr int T = 1024;         // threads of the listing kernels
constexpr int PER = 4;          // pages per thread
constexpr int CHUNK = T * PER;  // pages per CTA
constexpr int MAX_F = 65536;

// Workspace, in int32: head[4] (free pages, moved pages, 0, 0), counts[chunks],
// list_a[N], list_b[N], map[N], need[n].
struct Ws {
    int32_t *head, *counts, *list_a, *list_b, *map, *need;
    size_t bytes;
};
inline int chunks_of(int n_pages) { return (n_pages + CHUNK - 1) / CHUNK; }
Ws layout(void *base, int n_pages, int n) {
    Ws w{};
    int32_t *p = static_cast<int32_t *>(base);
    size_t off = 0;
    auto take = [&](size_t count) {
        int32_t *q = p + off;
        off += (count + 3) / 4 * 4;
        return q;
    };
    w.head = take(4);
    w.counts = take((size_t)chunks_of(n_pages));
    w.list_a = take((size_t)n_pages);
    w.list_b = take((size_t)n_pages);
    w.map = take((size_t)n_pages);
    w.need = take((size_t)n);
    w.bytes = off * sizeof(int32_t);
    return w;
}

// Sum over the CTA's threads, the same in all of them.
template <typename V>
__device__ __forceinline__ V block_sum(V v, V *smem) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) smem[threadIdx.x >> 5] = v;
    __syncthreads();
    V t = (threadIdx.x & 31) < (blockDim.x >> 5) ? smem[threadIdx.x & 31] : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(0xffffffffu, t, d);
    return t;
}
// Sum over the threads before this one; total receives the sum over all.
__device__ __forceinline__ int block_scan(int v, int *smem, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) smem[warp] = x;
    __syncthreads();
    int w = lane < (int)(blockDim.x >> 5) ? smem[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + x - v;
}

// Which of this thread's PER pages from p0 on are in use, as a bit mask (pages
// at or behind n count as not in use and not free).
__device__ __forceinline__ uint32_t live_mask(const int32_t *ref, int p0, int n) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < PER; i++)
        if (p0 + i < n && __ldg(ref + p0 + i) > 0) m |= 1u << i;
    return m;
}
__device__ __forceinline__ int valid_count(int p0, int n) {
    return p0 >= n ? 0 : (n - p0 < PER ? n - p0 : PER);
}

// Pages in use per chunk.
__global__ void __launch_bounds__(T) count_kernel(const int32_t *__restrict__ ref, int n, int32_t *counts) {
    __shared__ int smem[32];
    grid_dep_wait();
    grid_dep_launch();
    const int p0 = blockIdx.x * CHUNK + (int)threadIdx.x * PER;
    const int s = block_sum(__popc(live_mask(ref, p0, n)), smem);
    if (threadIdx.x == 0) counts[blockIdx.x] = s;
}

// Sum of counts[0, k) (and of all of them), by the whole CTA.
__device__ __forceinline__ int counts_before(const int32_t *counts, int k, int chunks, int &total, int *smem) {
    int a = 0, t = 0;
    for (int i = threadIdx.x; i < chunks; i += blockDim.x) {
        const int c = counts[i];
        t += c;
        if (i < k) a += c;
    }
    total = block_sum(t, smem);
    return block_sum(a, smem);
}

struct Fork {
    const int32_t *table;
    int S, max_pages, page_size, n_pages;
    const int64_t *seq_len;
    const int32_t *src, *dst;
    int F;
};
// Whole pages of a sequence's n tokens, and whether tokens remain behind them.
__device__ __forceinline__ void split_len(int64_t n, const Fork &f, int &full, bool &part) {
    const int64_t cap = (int64_t)f.max_pages * f.page_size;
    if (n < 0) n = 0;
    if (n > cap) n = cap;
    full = (int)(n / f.page_size);
    part = n % f.page_size != 0;
}
// By one warp: -1 fork i is refused, 1 it needs a page of its own, else 0.
__device__ int fork_need(const Fork &f, int i, int lane) {
    const int s = f.src[i], d = f.dst[i];
    if (s < 0 || s >= f.S || d < 0 || d >= f.S || s == d) return -1;
    bool bad = false;
    for (int k = lane; k < f.F; k += 32) {
        if (f.src[k] == d) bad = true;
        if (k < i && f.dst[k] == d) bad = true;
    }
    const int32_t *row = f.table + (int64_t)d * f.max_pages;
    for (int e = lane; e < f.max_pages; e += 32) {
        const int v = row[e];
        if (v >= 0 && v < f.n_pages) bad = true;
    }
    if (__any_sync(0xffffffffu, bad)) return -1;
    int full;
    bool part;
    split_len(f.seq_len[s], f, full, part);
    if (!part) return 0;
    const int last = f.table[(int64_t)s * f.max_pages + full];
    return last >= 0 && last < f.n_pages ? 1 : 0;
}

struct Extend {
    const int32_t *table;
    int S, max_pages, page_size, n_pages;
    const int64_t *want;
};
__device__ __forceinline__ int pages_of(int64_t n, int page_size, int max_pages) {
    if (n <= 0) return 0;
    const int64_t e = (n - 1) / page_size + 1;
    return e < max_pages ? (int)e : max_pages;
}
// By one warp: entries of sequence s that need a page.
__device__ int extend_need(const Extend &x, int s, int lane) {
    const int lim = pages_of(x.want[s], x.page_size, x.max_pages);
    const int32_t *row = x.table + (int64_t)s * x.max_pages;
    int c = 0;
    for (int e = lane; e < lim; e += 32) {
        const int v = row[e];
        c += v < 0 || v >= x.n_pages;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) c += __shfl_xor_sync(0xffffffffu, c, d);
    return c;
}

// Blocks [0, chunks): the free pages, ascending, to list, their number to
// head[0], and n_failed = 0. Blocks behind them: the needs, one warp each.
template <class R>
__global__ void __launch_bounds__(T)
    free_list_kernel(const int32_t *__restrict__ ref, int n, int chunks, const int32_t *counts, int32_t *head,
                     int32_t *list, R r, int n_req, int32_t *need, int32_t *n_failed) {
    __shared__ int smem[32];
    grid_dep_wait();
    grid_dep_launch();
    if ((int)blockIdx.x >= chunks) {
        const int i = ((int)blockIdx.x - chunks) * (T / 32) + (int)(threadIdx.x >> 5);
        if (i >= n_req) return;
        int v;
        if constexpr (std::is_same<R, Fork>::value)
            v = fork_need(r, i, threadIdx.x & 31);
        else
            v = extend_need(r, i, threadIdx.x & 31);
        if ((threadIdx.x & 31) == 0) need[i] = v;
        return;
    }
    const int c = blockIdx.x;
    int total = 0, before = 0;
    if (chunks > 1) before = counts_before(counts, c, chunks, total, smem);
    const int p0 = c * CHUNK + (int)threadIdx.x * PER;
    const uint32_t live = live_mask(ref, p0, n);
    const int valid = valid_count(p0, n);
    int own;
    const int rank = block_scan(valid - __popc(live), smem, own);
    int at = c * CHUNK - before + rank;  // free pages before p0
    for (int i = 0; i < valid; i++)
        if (!((live >> i) & 1)) list[at++] = p0 + i;
    if (c == 0 && threadIdx.x == 0) {
        head[0] = chunks > 1 ? n - total : own;
        *n_failed = 0;
    }
}

// ---------------------------------------------------------------- fork
constexpr int FT = 256;
__global__ void __launch_bounds__(FT)
    fork_kernel(int32_t *table, int32_t *ref, int64_t *seq_len, Fork f, const int32_t *head,
                const int32_t *list, const int32_t *need, int32_t *pairs, int32_t *n_failed) {
    __shared__ int smem[32];
    grid_dep_wait();
    grid_dep_launch();
    const int i = blockIdx.x;
    const int mine = need[i];
    const bool first = blockIdx.y == 0;
    if (mine < 0) {
        if (first && threadIdx.x == 0) {
            pairs[2 * i] = pairs[2 * i + 1] = -1;
            atomicAdd(n_failed, 1);
        }
        return;
    }
    const int s = f.src[i], d = f.dst[i];
    const int64_t n = seq_len[s];
    int full;
    bool part;
    split_len(n, f, full, part);
    const int32_t *from = table + (int64_t)s * f.max_pages;
    int32_t *to = table + (int64_t)d * f.max_pages;
    for (int e = blockIdx.y * FT + threadIdx.x; e < full; e += gridDim.y * FT) {
        const int v = from[e];
        const bool ok = v >= 0 && v < f.n_pages;
        to[e] = ok ? v : -1;
        if (ok) atomicAdd(ref + v, 1);
    }
    if (!first) return;
    int rank = 0;  // forks before this one that need a page
    if (mine) {
        for (int k = threadIdx.x; k < i; k += FT) rank += need[k] > 0;
        rank = block_sum(rank, smem);
    }
    if (threadIdx.x == 0) {
        int a = -1, b = -1;
        if (mine) {
            if (rank < head[0]) {
                a = from[full];
                b = list[rank];
                to[full] = b;
                ref[b] = 1;
            } else {
                atomicAdd(n_failed, 1);
            }
        }
        pairs[2 * i] = a;
        pairs[2 * i + 1] = b;
        seq_len[d] = mine && b < 0 ? (int64_t)full * f.page_size : n;
    }
}

// ---------------------------------------------------------------- extend
// Needs are summed in 64 bits: a table may lack more than 2^31 pages. What fails is
// what is needed beyond the free pages; the last sequence's block counts it.
__global__ void __launch_bounds__(FT)
    extend_kernel(int32_t *table, int32_t *ref, Extend x, const int32_t *head, const int32_t *list,
                  const int32_t *need, int32_t *n_failed) {
    __shared__ int smem[32];
    __shared__ int64_t wide[32];
    grid_dep_wait();
    grid_dep_launch();
    const int s = blockIdx.x, own = need[s];
    const bool last = s == x.S - 1;
    if (own == 0 && !last) return;
    int64_t before = 0;  // entries of earlier sequences that need a page
    for (int k = threadIdx.x; k < s; k += FT) before += need[k];
    before = block_sum(before, wide);
    const int n_free = head[0];
    if (last && threadIdx.x == 0) {
        const int64_t failed = before + own - n_free;
        *n_failed = failed <= 0 ? 0 : failed < INT32_MAX ? (int32_t)failed : INT32_MAX;
    }
    if (own == 0) return;
    const int lim = pages_of(x.want[s], x.page_size, x.max_pages);
    int32_t *row = table + (int64_t)s * x.max_pages;
    for (int e0 = 0; e0 < lim; e0 += FT) {
        const int e = e0 + (int)threadIdx.x;
        bool miss = false;
        if (e < lim) {
            const int v = row[e];
            miss = v < 0 || v >= x.n_pages;
        }
        int total;
        const int64_t rank = before + block_scan(miss, smem, total);
        before += total;
        if (miss && rank < n_free) {
            const int p = list[rank];
            row[e] = p;
            ref[p] = 1;
        }
    }
}

// ---------------------------------------------------------------- free
__global__ void __launch_bounds__(FT)
    free_kernel(int32_t *table, int S, int max_pages, int32_t *ref, int n_pages, int page_size,
                const int32_t *__restrict__ seq, const int64_t *__restrict__ keep_len) {
    grid_dep_wait();
    grid_dep_launch();
    const int s = seq[blockIdx.x];
    if (s < 0 || s >= S) return;
    const int keep = keep_len ? pages_of(keep_len[blockIdx.x], page_size, max_pages) : 0;
    int32_t *row = table + (int64_t)s * max_pages;
    for (int e = keep + (int)(blockIdx.y * FT + threadIdx.x); e < max_pages; e += gridDim.y * FT) {
        // exchanged, so that a sequence listed twice gives a page back once
        const int v = atomicExch(row + e, -1);
        if (v >= 0 && v < n_pages) atomicSub(ref + v, 1);
    }
}

// ---------------------------------------------------------------- copies
// Pages are cut into units of UNIT bytes (the last of a page shorter); a CTA
// takes whole units, 16 bytes per thread and access, all loads of a unit before
// its stores.
constexpr int CT = 256;
constexpr int IN_FLIGHT = 4;
constexpr int UNIT = CT * IN_FLIGHT * 16;
struct Bufs {
    uint8_t *base[CSA2_MAX_PAGE_BUFS];
    int64_t bytes[CSA2_MAX_PAGE_BUFS];
    int width[CSA2_MAX_PAGE_BUFS];   // access width: 16, 4 or 1
    int64_t unit0[CSA2_MAX_PAGE_BUFS + 1];  // units of a page before buffer k
    int n;
};

template <typename W>
__device__ __forceinline__ void copy_unit(const uint8_t *src, uint8_t *dst, int bytes) {
    const W *s = reinterpret_cast<const W *>(src);
    W *d = reinterpret_cast<W *>(dst);
    const int n = bytes / (int)sizeof(W);
    for (int i0 = threadIdx.x; i0 < n; i0 += CT * IN_FLIGHT) {
        W v[IN_FLIGHT];
#pragma unroll
        for (int k = 0; k < IN_FLIGHT; k++)
            if (i0 + k * CT < n) v[k] = s[i0 + k * CT];
#pragma unroll
        for (int k = 0; k < IN_FLIGHT; k++)
            if (i0 + k * CT < n) d[i0 + k * CT] = v[k];
    }
}

// Unit u of page src onto page dst.
__device__ __forceinline__ void copy_page_unit(const Bufs &b, int src, int dst, int64_t u) {
    int k = 0;
    while (k + 1 < b.n && u >= b.unit0[k + 1]) k++;
    const int64_t off = (u - b.unit0[k]) * UNIT, left = b.bytes[k] - off;
    const int bytes = left < UNIT ? (int)left : UNIT;
    const uint8_t *s = b.base[k] + (int64_t)src * b.bytes[k] + off;
    uint8_t *d = b.base[k] + (int64_t)dst * b.bytes[k] + off;
    if (b.width[k] == 16)
        copy_unit<uint4>(s, d, bytes);
    else if (b.width[k] == 4)
        copy_unit<uint32_t>(s, d, bytes);
    else
        copy_unit<uint8_t>(s, d, bytes);
}

__global__ void __launch_bounds__(CT)
    copy_kernel(const int32_t *__restrict__ pairs, int F, int n_pages, const __grid_constant__ Bufs b) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t per = b.unit0[b.n], total = per * F;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int f = (int)(i / per);
        const int src = __ldg(pairs + 2 * f), dst = __ldg(pairs + 2 * f + 1);
        if (src < 0 || src >= n_pages || dst < 0 || dst >= n_pages || src == dst) continue;
        copy_page_unit(b, src, dst, i - f * per);
    }
}

// ---------------------------------------------------------------- compact
// With L pages in use: hole i = the i-th free page before L, mover i = the i-th
// page in use from L on; there are as many of one as of the other. map[p] of a
// mover is its i.
__global__ void __launch_bounds__(T)
    compact_list_kernel(const int32_t *__restrict__ ref, int n, int chunks, const int32_t *counts, int32_t *head,
                        int32_t *holes, int32_t *movers, int32_t *map, int32_t *n_live) {
    __shared__ int smem[32];
    grid_dep_wait();
    grid_dep_launch();
    const int c = blockIdx.x;
    const int p0 = c * CHUNK + (int)threadIdx.x * PER;
    const uint32_t live = live_mask(ref, p0, n);
    int own;
    const int rank = block_scan(__popc(live), smem, own);
    int L = own, before = 0, below;  // below: pages in use before L
    if (chunks > 1) {
        before = counts_before(counts, c, chunks, L, smem);
        int unused;
        const int cl = L / CHUNK;  // the chunk that L falls in
        below = counts_before(counts, cl, chunks, unused, smem);
        const int q0 = cl * CHUNK + (int)threadIdx.x * PER;
        uint32_t m = live_mask(ref, q0, n);
        const int first = L - q0;  // of this thread's pages, those before L
        m = first <= 0 ? 0u : (first < PER ? m & ((1u << first) - 1) : m);
        below += block_sum(__popc(m), smem);
    } else {
        const int first = L - p0;
        const uint32_t m = first <= 0 ? 0u : (first < PER ? live & ((1u << first) - 1) : live);
        below = block_sum(__popc(m), smem);
    }
    int r = before + rank;  // pages in use before p
    const int valid = valid_count(p0, n);
    for (int i = 0; i < valid; i++) {
        const int p = p0 + i;
        const bool in_use = (live >> i) & 1;
        if (!in_use && p < L) holes[p - r] = p;
        if (in_use && p >= L) {
            movers[r - below] = p;
            map[p] = r - below;
        }
        r += in_use;
    }
    if (c == 0 && threadIdx.x == 0) {
        head[0] = L;
        head[1] = L - below;
        *n_live = L;
    }
}

__global__ void __launch_bounds__(CT)
    compact_apply_kernel(const int32_t *table, int64_t entries, const int32_t *ref, int n, const int32_t *head,
                         const int32_t *holes, const int32_t *movers, const int32_t *map, int32_t *table_out,
                         int32_t *ref_out, const __grid_constant__ Bufs b) {
    grid_dep_wait();
    grid_dep_launch();
    const int L = head[0], moves = head[1];
    const int64_t tid = (int64_t)blockIdx.x * CT + threadIdx.x, all = (int64_t)gridDim.x * CT;
    // a hole's thread also clears its mover's place, so that in place nobody
    // reads a count that another thread has cleared
    for (int64_t p = tid; p < n; p += all) {
        const int c = ref[p];
        if (p >= L) {
            if (c <= 0) ref_out[p] = 0;
        } else if (c > 0) {
            ref_out[p] = c;
        }
    }
    for (int64_t i = tid; i < moves; i += all) {
        ref_out[holes[i]] = ref[movers[i]];
        ref_out[movers[i]] = 0;
    }
    for (int64_t i = tid; i < entries; i += all) {
        const int v = table[i];
        int o = v;
        // map holds a value for the pages that move alone
        if (v >= L && v < n) {
            const int m = map[v];
            if (m >= 0 && m < moves && movers[m] == v) o = holes[m];
        }
        table_out[i] = o;
    }
    if (b.n == 0) return;
    const int64_t per = b.unit0[b.n], total = per * moves;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int m = (int)(i / per);
        copy_page_unit(b, movers[m], holes[m], i - m * per);
    }
}

// ---------------------------------------------------------------- host side
int make_bufs(const csa2_page_buf *bufs, int n, Bufs &b) {
    b = Bufs{};
    b.n = n;
    for (int k = 0; k < n; k++) {
        if (!bufs[k].base) return CSA2_ERR_NULL;
        if (bufs[k].page_bytes < 1 || bufs[k].page_bytes >= (1ll << 40)) return CSA2_ERR_SHAPE;
        b.base[k] = static_cast<uint8_t *>(bufs[k].base);
        b.bytes[k] = bufs[k].page_bytes;
        const uint64_t bits = reinterpret_cast<uintptr_t>(bufs[k].base) | (uint64_t)bufs[k].page_bytes;
        b.width[k] = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
        b.unit0[k + 1] = b.unit0[k] + (bufs[k].page_bytes + UNIT - 1) / UNIT;
    }
    return CSA2_OK;
}

bool table_ok(int S, int max_pages, int page_size, int n_pages) {
    return S >= 0 && paged_shape_ok(max_pages, page_size, n_pages);
}

// The blocks of a row's entries: a few entries per thread.
unsigned row_blocks(int max_pages) {
    const int b = (max_pages + FT * 4 - 1) / (FT * 4);
    return (unsigned)(b < 1 ? 1 : b > 1024 ? 1024 : b);
}

template <class R>
int free_list(const int32_t *ref, int n_pages, const Ws &w, const R &r, int n_req, int32_t *n_failed,
              cudaStream_t s) {
    const int chunks = chunks_of(n_pages);
    if (chunks > 1) {
        const int st = launch_kernel(true, count_kernel, dim3((unsigned)chunks), dim3(T), 0, s, ref, n_pages,
                                     w.counts);
        if (st != CSA2_OK) return st;
    }
    const unsigned grid = (unsigned)(chunks + (n_req + T / 32 - 1) / (T / 32));
    return launch_kernel(true, free_list_kernel<R>, dim3(grid), dim3(T), 0, s, ref, n_pages, chunks,
                         (const int32_t *)w.counts, w.head, w.list_a, r, n_req, w.need, n_failed);
}

}  // namespace pages
}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_pages_workspace_size(int n_pages, int n) {
    if (n_pages < 1 || n_pages > MAX_PAGES || n < 0) return 0;
    return pages::layout(nullptr, n_pages, n).bytes;
}

extern "C" int csa2_pages_extend(int32_t *page_table, int S, int max_pages, int32_t *ref, int n_pages,
                                 int page_size, const int64_t *want_len, int32_t *n_failed, void *ws,
                                 size_t ws_bytes, void *stream) {
    if (!ref || !n_failed || (S != 0 && (!page_table || !want_len))) return CSA2_ERR_NULL;
    if (!pages::table_ok(S, max_pages, page_size, n_pages)) return CSA2_ERR_SHAPE;
    const pages::Ws w = pages::layout(ws, n_pages, S);
    if (!ws || ws_bytes < w.bytes) return CSA2_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return CSA2_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const pages::Extend x{page_table, S, max_pages, page_size, n_pages, want_len};
    int st = pages::free_list(ref, n_pages, w, x, S, n_failed, s);
    if (st != CSA2_OK || S == 0) return st;
    return launch_kernel(true, pages::extend_kernel, dim3((unsigned)S), dim3(pages::FT), 0, s, page_table, ref, x,
                         (const int32_t *)w.head, (const int32_t *)w.list_a, (const int32_t *)w.need, n_failed);
}

extern "C" int csa2_pages_fork(int32_t *page_table, int S, int max_pages, int32_t *ref, int n_pages,
                               int page_size, int64_t *seq_len, const int32_t *src, const int32_t *dst,
                               int F, int32_t *pairs, int32_t *n_failed, void *ws, size_t ws_bytes,
                               void *stream) {
    if (!ref || !n_failed || (F != 0 && (!page_table || !seq_len || !src || !dst || !pairs)))
        return CSA2_ERR_NULL;
    if (!pages::table_ok(S, max_pages, page_size, n_pages) || F < 0 || F > pages::MAX_F) return CSA2_ERR_SHAPE;
    const pages::Ws w = pages::layout(ws, n_pages, F);
    if (!ws || ws_bytes < w.bytes) return CSA2_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return CSA2_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const pages::Fork f{page_table, S, max_pages, page_size, n_pages, seq_len, src, dst, F};
    int st = pages::free_list(ref, n_pages, w, f, F, n_failed, s);
    if (st != CSA2_OK || F == 0) return st;
    return launch_kernel(true, pages::fork_kernel, dim3((unsigned)F, pages::row_blocks(max_pages)),
                         dim3(pages::FT), 0, s, page_table, ref, seq_len, f, (const int32_t *)w.head,
                         (const int32_t *)w.list_a, (const int32_t *)w.need, pairs, n_failed);
}

extern "C" int csa2_pages_free(int32_t *page_table, int S, int max_pages, int32_t *ref, int n_pages,
                               int page_size, const int32_t *seq, const int64_t *keep_len, int F,
                               void *stream) {
    if (F != 0 && (!page_table || !ref || !seq)) return CSA2_ERR_NULL;
    if (!pages::table_ok(S, max_pages, page_size, n_pages) || F < 0) return CSA2_ERR_SHAPE;
    if (F == 0) return CSA2_OK;
    return launch_kernel(true, pages::free_kernel, dim3((unsigned)F, pages::row_blocks(max_pages)),
                         dim3(pages::FT), 0, (cudaStream_t)stream, page_table, S, max_pages, ref, n_pages,
                         page_size, seq, keep_len);
}

extern "C" int csa2_pages_copy(const int32_t *pairs, int F, const csa2_page_buf *bufs, int n_bufs,
                               int n_pages, void *stream) {
    if (!bufs || (F != 0 && !pairs)) return CSA2_ERR_NULL;
    if (F < 0 || n_pages < 1 || n_bufs < 1 || n_bufs > CSA2_MAX_PAGE_BUFS) return CSA2_ERR_SHAPE;
    pages::Bufs b;
    const int st = pages::make_bufs(bufs, n_bufs, b);
    if (st != CSA2_OK) return st;
    if (F == 0) return CSA2_OK;
    const int64_t units = b.unit0[n_bufs] * F, most = (int64_t)num_sms() * 8;
    return launch_kernel(true, pages::copy_kernel, dim3((unsigned)(units < most ? units : most)),
                         dim3(pages::CT), 0, (cudaStream_t)stream, pairs, F, n_pages, b);
}

extern "C" int csa2_pages_compact(const int32_t *page_table, int S, int max_pages, const int32_t *ref,
                                  int n_pages, const csa2_page_buf *bufs, int n_bufs,
                                  int32_t *page_table_out, int32_t *ref_out, int32_t *n_live, void *ws,
                                  size_t ws_bytes, void *stream) {
    if (!ref || !ref_out || !n_live || (S != 0 && (!page_table || !page_table_out)) || (n_bufs > 0 && !bufs))
        return CSA2_ERR_NULL;
    if (!pages::table_ok(S, max_pages, 1, n_pages) || n_bufs < 0 || n_bufs > CSA2_MAX_PAGE_BUFS)
        return CSA2_ERR_SHAPE;
    pages::Bufs b;
    int st = pages::make_bufs(bufs, n_bufs, b);
    if (st != CSA2_OK) return st;
    const pages::Ws w = pages::layout(ws, n_pages, 0);
    if (!ws || ws_bytes < w.bytes) return CSA2_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return CSA2_ERR_ALIGN;
    cudaStream_t s = (cudaStream_t)stream;
    const int chunks = pages::chunks_of(n_pages);
    if (chunks > 1) {
        st = launch_kernel(true, pages::count_kernel, dim3((unsigned)chunks), dim3(pages::T), 0, s, ref, n_pages,
                           w.counts);
        if (st != CSA2_OK) return st;
    }
    st = launch_kernel(true, pages::compact_list_kernel, dim3((unsigned)chunks), dim3(pages::T), 0, s, ref,
                       n_pages, chunks, (const int32_t *)w.counts, w.head, w.list_a, w.list_b, w.map, n_live);
    if (st != CSA2_OK) return st;
    const int64_t entries = (int64_t)S * max_pages;
    // enough CTAs for the copies, fewer when there is only a table to rewrite
    int64_t grid = n_bufs ? b.unit0[n_bufs] * (n_pages / 2) : 0;
    const int64_t flat = (entries + n_pages + pages::CT * 4 - 1) / (pages::CT * 4);
    if (grid < flat) grid = flat;
    if (grid > (int64_t)num_sms() * 8) grid = (int64_t)num_sms() * 8;
    return launch_kernel(true, pages::compact_apply_kernel, dim3((unsigned)grid), dim3(pages::CT), 0, s, page_table,
                         entries, ref, n_pages, (const int32_t *)w.head, (const int32_t *)w.list_a,
                         (const int32_t *)w.list_b, (const int32_t *)w.map, page_table_out, ref_out, b);
}
