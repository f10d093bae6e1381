// ssu_paged.cpp -- host side of the paged cache's kernels: how a call is
// computed, tensor maps, device properties.
#include "ssu_paged.h"

#include "ssu.h"

namespace ssu {

namespace {

// The driver's tensor-map encoder, looked up once.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

}  // namespace

namespace {

bool encode_boxes(CUtensorMap *m, const PagedParams &p, const void *base, const int64_t *stride, int tokens, bool both) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    // [element, row, half, head, page]
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(both ? 64 : p.D), static_cast<cuuint64_t>(p.page), both ? 2u : 1u,
                                static_cast<cuuint64_t>(p.G), static_cast<cuuint64_t>(p.pages)};
    // a stride along an extent of one is never used: keep it legal
    const int64_t at[4] = {stride[1], both ? 64 : p.D, p.G > 1 ? stride[2] : p.D, p.pages > 1 ? stride[0] : p.D};
    cuuint64_t strides[4];
    for (int i = 0; i < 4; ++i) strides[i] = static_cast<cuuint64_t>(at[i]) * 2;
    const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(tokens), both ? 2u : 1u, 1, 1}, unit[5] = {1, 1, 1, 1, 1};
    const CUtensorMapDataType type = p.io_dtype == SSU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, type, 5, const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int least_box(const PagedParams &p, int keys) {
    int least = keys;
    while (p.page % least != 0) least /= 2;
    return least;
}

bool encode_cache(CacheMaps *m, const PagedParams &p, int keys) {
    const int least = least_box(p, keys);
    for (int i = 0; i < kBoxes; ++i) {
        const int tokens = 8 << i;
        if (tokens < least) continue;
        if (tokens > keys || tokens > p.page) break;
        const bool both = tokens == keys && p.D == 128;
        if (!encode_boxes(&m->k[i], p, p.k_cache, p.ks, tokens, both) || !encode_boxes(&m->v[i], p, p.v_cache, p.vs, tokens, both))
            return false;
    }
    return true;
}

bool encode_queries(CUtensorMap *m, const PagedParams &p, int tokens) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.D), static_cast<cuuint64_t>(p.H), static_cast<cuuint64_t>(p.rows)};
    const int64_t hs = p.H > 1 ? p.qs[1] : p.D, ts = p.rows > 1 ? p.qs[0] : p.D;
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2, static_cast<cuuint64_t>(ts) * 2};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(p.share), static_cast<cuuint32_t>(tokens)}, unit[3] = {1, 1, 1};
    const CUtensorMapDataType type = p.io_dtype == SSU_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, type, 3, const_cast<void *>(p.q), dims, strides, boxes, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int device_sms() {
    static int cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    int *const kept = dev >= 0 && dev < 64 ? &cache[dev] : nullptr;
    int n = kept ? __atomic_load_n(kept, __ATOMIC_RELAXED) : 0;
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        if (kept) __atomic_store_n(kept, n, __ATOMIC_RELAXED);
    }
    return n;
}

// By the rows (new tokens x heads on a key/value head) of the longest sequence.
// Up to 64 go to the kernel for few rows, which reads every key once for 16, 32
// or 64 of them: 32 sequences of 5 drafts, 20 / 4 heads of 96 (25 rows), 54 us,
// where tiles of 128 rows take 80.  More go to the tiles, single tokens among
// them too: taken to the other kernel first, three quarters of a batch of 43
// made 281 us of 233.
AttendPlan attend_plan(const AttendParams &p, int64_t max_seqlen, int64_t max_kv_len) {
    AttendPlan a{};
    a.max_kv_len = max_kv_len;
    const int64_t given = max_seqlen < p.c.rows ? max_seqlen : p.c.rows;  // (no sequence is longer)
    const int64_t longest = p.c.cu == nullptr ? 1 : max_seqlen > 0 ? given : (p.c.rows + p.c.nseq - 1) / p.c.nseq;
    const int64_t rows = longest * p.c.share;
    a.kind = rows <= 16 ? kAttendRows16 : rows <= 32 ? kAttendRows32 : rows <= 64 ? kAttendRows64 : kAttendTiles;
    a.bytes = a.kind == kAttendTiles ? attend_tiles_workspace(p.c, max_kv_len) : attend_rows_workspace(a.kind, p.c.D);
    return a;
}

cudaError_t launch_paged_attention(const AttendParams &p, const AttendPlan &plan, void *workspace, cudaStream_t stream) {
    if (plan.kind == kAttendTiles) return launch_attend_tiles(p, plan.max_kv_len, workspace, stream);
    return launch_attend_rows(p, plan.kind, workspace, stream);
}

}  // namespace ssu
