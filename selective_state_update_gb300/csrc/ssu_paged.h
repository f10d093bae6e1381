// ssu_paged.h -- parameters shared by the host layer and the kernels of the
// paged key / value cache: appending to it and attention over it.  Not part of
// the public ABI (that is include/ssu.h).
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

namespace ssu {

// Sequence b has the rows [cu[b], cu[b + 1]) (row b without cu) of the new
// tokens, the last ones of its kv_lens[b] tokens; key j of it lies in page
// table[b][j / page], row j % page.  Strides are in elements, the innermost is
// one: [page, row, head] of the caches, [row, head] of q and out.
struct PagedParams {
    int64_t pages, rows, nseq;
    int32_t page;              // tokens of a page
    int32_t H, G, share, D;    // heads, key/value heads, heads / key/value heads, head size
    int32_t io_dtype;
    int32_t table_is_i64, meta_is_i64;
    void *k_cache, *v_cache;
    int64_t ks[3], vs[3];
    const void *table;
    int64_t table_stride, table_width;
    const void *kv_lens, *cu;
    const void *q;
    void *out;
    int64_t qs[2], os[2];
    int32_t *status;
};
constexpr int kPagedMaxDim = 128;      // largest head size
constexpr int kPagedMaxShare = 128;    // most heads on one key/value head
constexpr int64_t kPagedMaxLen = 1 << 30;  // longest sequence

struct AppendParams {
    PagedParams c;  // q -> out (rotated), or out == nullptr: no q
    const void *k, *v;
    int64_t kstr[2], vstr[2];
    const float *inv_freq;  // nullptr: no rotation
    int32_t rotary, interleaved;
};
cudaError_t launch_paged_append(const AppendParams &p, cudaStream_t stream);

struct AttendParams {
    PagedParams c;
    float scale;       // positive
    int32_t window;    // 0: all earlier keys
    float *lse;        // [rows, H] or nullptr
};
// How a call is computed, and the workspace it needs for that.
struct AttendPlan {
    int32_t kind;      // kAttendRows*, kAttendTiles
    int64_t max_kv_len;
    uint64_t bytes;
};
enum : int32_t { kAttendRows16 = 0, kAttendRows32 = 1, kAttendRows64 = 2, kAttendTiles = 3 };
AttendPlan attend_plan(const AttendParams &p, int64_t max_seqlen, int64_t max_kv_len);
cudaError_t launch_paged_attention(const AttendParams &p, const AttendPlan &plan, void *workspace, cudaStream_t stream);
cudaError_t launch_attend_rows(const AttendParams &p, int kind, void *workspace, cudaStream_t stream);
uint64_t attend_rows_workspace(int kind, int D);
cudaError_t launch_attend_tiles(const AttendParams &p, int64_t max_kv_len, void *workspace, cudaStream_t stream);
uint64_t attend_tiles_workspace(const PagedParams &c, int64_t max_kv_len);

// The tensor maps of a cache: map i has boxes of 8 << i tokens of one head by
// 64 elements or, where it is as high as a tile of keys and the head size is 128,
// by both halves of that.  A tile of keys
// is copied in the largest boxes that the pages' ends allow: boxes of the
// largest power of two that divides the page instead (16 tokens for pages of 272)
// took 1065 us where these took 885 (2048 tokens behind 72000, 16 / 4 heads of 128).
constexpr int kBoxes = 5;
struct CacheMaps {
    CUtensorMap k[kBoxes], v[kBoxes];
};
// Tiles begin at multiples of `keys` tokens, so the distance to a page's end is a
// multiple of the largest power of two that divides both; what a tile needs is rounded to that.
int least_box(const PagedParams &p, int keys);
// Maps of the boxes that tiles of `keys` tokens need.
bool encode_cache(CacheMaps *m, const PagedParams &p, int keys);
// ... and of the queries: boxes of `tokens` tokens by the heads of a group by 64 elements.
bool encode_queries(CUtensorMap *m, const PagedParams &p, int tokens);
int device_sms();

}  // namespace ssu
