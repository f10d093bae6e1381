// ssu_paged.cuh -- device code shared by the kernels of the paged cache: a
// sequence's metadata, the cache's tiled copies, products of 16 x 8 x 16.
#pragma once

#include "ssu_device.cuh"
#include "ssu_paged.h"

namespace ssu {

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

// The page that holds tokens from `token` on of sequence b, or -1 (flagged)
// where the table names none.
__device__ __forceinline__ int64_t page_of(const PagedParams &p, int64_t b, int32_t token) {
    const int64_t page = load_index(p.table, b * p.table_stride + token / p.page, p.table_is_i64);
    if (page >= 0 && page < p.pages) return page;
    flag(p.status, kDevBadSlot);
    return -1;
}

// Tiled copy global -> shared of a 4-D box, completed on `bar`.  x * element
// size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(void *dst_smem, const void *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            smem_addr(dst_smem)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// True where 16 bytes of 16-bit floats hold an infinity or a NaN.
template <bool BF>
__device__ __forceinline__ bool any_odd(const uint4 &v) {
    constexpr uint32_t kExp = BF ? 0x7f80u : 0x7c00u;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t u = (&v.x)[i];
        odd = odd || (u & kExp) == kExp || ((u >> 16) & kExp) == kExp;
    }
    return odd;
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
