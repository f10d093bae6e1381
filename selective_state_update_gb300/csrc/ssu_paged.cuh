// ssu_paged.cuh -- device code shared by the kernels of the paged cache: a
// sequence's metadata, the cache's tiled copies, products of 16 x 8 x 16.
#pragma once

#include <utility>

#include "ssu_paged.h"
#include "ssu_tcgen05.cuh"

namespace ssu {

// A kernel that is launched to start while the one before it on the stream ends:
// it waits here until that has ended and what it wrote is there.
__device__ __forceinline__ void wait_for_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// ... which lets it start, once all of its CTAs have come here.
__device__ __forceinline__ void start_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Args, typename... Given>
cudaError_t launch_after(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Given &&...args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid, config.blockDim = dim3(threads), config.dynamicSmemBytes = smem, config.stream = stream;
    config.attrs = &attr, config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, kernel, std::forward<Given>(args)...);
}

struct Seq {
    int64_t t0;  // first row of its new tokens
    int32_t n;   // new tokens; 0 as well where the sequence is to be skipped
    int32_t kv;  // tokens in the cache, the new ones among them
};

// Sequence b's metadata, checked; n = 0 (and flagged) where it is bad.
__device__ __forceinline__ Seq load_seq(const PagedParams &p, int64_t b, bool report) {
    int64_t t0 = b, t1 = b + 1;
    if (p.cu != nullptr) t0 = load_index(p.cu, b, p.meta_is_i64), t1 = load_index(p.cu, b + 1, p.meta_is_i64);
    const int64_t kv = load_index(p.kv_lens, b, p.meta_is_i64);
    Seq s{t0, 0, 0};
    if (t0 < 0 || t1 < t0 || t1 > p.rows || kv < 0 || kv > kPagedMaxLen || kv > p.table_width * p.page) {
        if (report) flag(p.status, kDevBadSeqlen);
        return s;
    }
    s.n = static_cast<int32_t>(t1 - t0);
    s.kv = static_cast<int32_t>(kv);
    return s;
}

// Sequence b's page `i`, or -1 (flagged) where the table names none.
__device__ __forceinline__ int64_t table_page(const PagedParams &p, int64_t b, int32_t i) {
    const int64_t page = load_index(p.table, b * p.table_stride + i, p.table_is_i64);
    if (page >= 0 && page < p.pages) return page;
    flag(p.status, kDevBadSlot);
    return -1;
}
// The page of sequence b that holds its token `token`.
__device__ __forceinline__ int64_t page_of(const PagedParams &p, int64_t b, int32_t token) { return table_page(p, b, token / p.page); }

// Tiled copy global -> shared of a 5-D box, completed on `bar`.  x * element
// size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_5d(uint32_t dst_smem, const void *map, int x, int y, int z, int u, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(
            dst_smem),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(u), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Division by a page's length: by its reciprocal, rounded down, which is at most
// one too small for numbers below 2^30.
struct PageDivider {
    uint32_t page, inverse;
    __device__ __forceinline__ explicit PageDivider(int p) : page(p), inverse(0xffffffffu / static_cast<uint32_t>(p)) {}
    __device__ __forceinline__ int divide(int n, int &rest) const {
        uint32_t q = __umulhi(static_cast<uint32_t>(n), inverse), r = static_cast<uint32_t>(n) - q * page;
        if (r >= page) ++q, r -= page;
        rest = static_cast<int>(r);
        return static_cast<int>(q);
    }
};

// Copies tiles of KEYS keys or values, PANELS x 64 elements wide, from their
// pages, a lane each box.  What there is to copy is found ahead of the wait for a
// place to put it, with little arithmetic: one warp does it, an instruction at a
// time.  (With divisions and the general case for every tile, single tokens took
// 1.6 us a tile of 64 keys on every CTA whatever its size.)
template <int KEYS, int PANELS>
struct PageCopier {
    static constexpr int kPanelBytes = KEYS * 128;
    const PagedParams &p;
    int least;  // what tiles are rounded to
    PageDivider by_page;
    bool regular;              // every box of a tile is `least` rows of a page of its own, or the tile lies within one page
    int box, x, at, dst;       // this lane's box where that is so: its map, element, first row of the tile; where it goes
    struct Tile {
        uint32_t bytes;
        int page;        // this lane's: entry `first` + lane of the table; where regular, its box's
        int box, x, y;   // this lane's box: its map (-1: none), element, row of the page
        int entry, dst;  // ... whose page which lane has, and where it goes
    };
    __device__ __forceinline__ PageCopier(const PagedParams &params, int least_rows)
        : p(params), least(least_rows), by_page(params.page) {
        const int lane = threadIdx.x & 31;
        regular = least == KEYS || least == p.page;
        const int halves = PANELS == 2 && !(least == KEYS && p.D == 128) ? 2 : 1, half = lane % halves;
        at = lane / halves * least;
        box = at < KEYS ? 28 - __clz(least) : -1;
        x = 64 * half;
        dst = half * kPanelBytes + at * 128;
    }
    // The rows [from, to) of tile j that some query sees, where it sees the keys [lo, end).
    __device__ __forceinline__ void rows(int j, int lo, int end, int &from, int &to) const {
        to = min((max(end - j * KEYS, 0) + least - 1) & -least, KEYS);
        from = min(max(lo - j * KEYS, 0) & -least, to);
    }
    // This lane's page of tile j of sequence b; the number is on its way when
    // this returns.
    __device__ __forceinline__ int look_up(int64_t b, int j, int lo, int end) const {
        int from, to, rest;
        rows(j, lo, end, from, to);
        int entry;
        if (regular) {
            entry = by_page.divide(j * KEYS + at, rest);
            if (at < from || at >= to) return 0;
        } else {
            entry = by_page.divide(j * KEYS + from, rest) + (threadIdx.x & 31);
            if (to <= from || entry * static_cast<int64_t>(p.page) >= j * KEYS + to) return 0;
        }
        const int64_t page = table_page(p, b, entry);
        return static_cast<int>(page < 0 ? p.pages : page);  // past the last page the copies read zeros
    }
    // What tile j takes, its pages looked up.
    __device__ __forceinline__ Tile find(int page, int j, int lo, int end) const {
        const int lane = threadIdx.x & 31;
        int from, to;
        rows(j, lo, end, from, to);
        Tile t;
        t.bytes = static_cast<uint32_t>(to - from) * (128 * PANELS);
        t.page = page;
        if (regular) {
            by_page.divide(j * KEYS + at, t.y);
            t.box = at >= from && at < to ? box : -1, t.x = x, t.entry = lane, t.dst = dst;
            return t;
        }
        t.box = -1, t.x = 0, t.y = 0, t.entry = 0, t.dst = 0;
        int y;
        by_page.divide(j * KEYS + from, y);
        // the largest boxes that the pages' ends allow: 32 at most, as many as pages of 8 tokens take
#pragma unroll 1
        for (int row = from, entry = 0, op = 0; row < to;) {
            const int h = 31 - __clz(min(min(to - row, p.page - y), KEYS)), count = 1 << h;
            // (a box of KEYS rows has both halves of 128 elements)
            const int ops = PANELS == 2 && !(count == KEYS && p.D == 128) ? 2 : 1;
            if (lane >= op && lane < op + ops) {
                const int half = lane - op;
                t.box = h - 3, t.x = 64 * half, t.y = y, t.entry = entry, t.dst = half * kPanelBytes + row * 128;
            }
            op += ops, row += count, y += count;
            if (y == p.page) y = 0, ++entry;
        }
        return t;
    }
    __device__ __forceinline__ void copy(const Tile &t, const CUtensorMap *maps, int g, uint32_t to, uint64_t *bar) const {
        const int page = __shfl_sync(0xffffffffu, t.page, t.entry);
        if (t.box >= 0) tma_load_5d(to + t.dst, maps + t.box, t.x, t.y, 0, g, page, bar);
        __syncwarp();
    }
};

// True where 16 bytes of 16-bit floats hold an infinity or a NaN: a sum of zeros
// times them is no zero.
template <bool BF>
__device__ __forceinline__ bool any_odd(const uint4 &v) {
    uint32_t sum = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"((&v.x)[i]), "r"(0u));
        else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"((&v.x)[i]), "r"(0u));
    }
    return (sum & 0x7fff7fffu) != 0u;
}
// The same 16 bytes with zeros for them.
template <bool BF>
__device__ __forceinline__ uint4 without_odd(uint4 v) {
    constexpr uint32_t kExp = BF ? 0x7f80u : 0x7c00u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t &u = (&v.x)[i];
        if ((u & kExp) == kExp) u &= 0xffff0000u;
        if (((u >> 16) & kExp) == kExp) u &= 0x0000ffffu;
    }
    return v;
}

}  // namespace ssu
