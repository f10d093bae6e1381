// ssu_paged_rows.cu -- attention over the paged cache for few query rows: single
// tokens and drafts.
//
// A tile is 16, 32 or 64 query rows of one sequence that share a key/value head --
// row m of the sequence is token m / share, head m % share of the group -- and
// 64 keys.  One pass over the keys with a running maximum and sum:
//     x_j = scale log2(e) q . k_j,  m' = max(m, x_j),
//     l' = l 2^(m - m') + sum_j 2^(x_j - m'),  o' = o 2^(m - m') + sum_j 2^(x_j - m') v_j
// and out = o / l, lse = (m + log2 l) ln 2, all of it in fp32; P = 2^(x - m') is
// rounded once to the io type, as the product's operand.  For fp16 m is the maximum
// less 15 (kLift), so that P goes up to 2^15 and is rounded by half a step down to 2^-29 of
// the largest weight, and by 2^-40 of it below: without, the tokens of a long context
// beside one that takes nearly all the weight, 2^-25 of it each, were nothing.
//
// Bound by HBM: a key and its value are 4 D bytes and 4 D share operations.  So
// what counts is that every SM reads all the time, whatever the lengths: all
// (sequence, row tile, head, key tile) of the call are numbered in this order
// and every CTA takes an equal share of the numbers, cut anywhere.  A CTA that
// has a whole run of one row tile's keys stores its outputs; where the run is
// cut, (o, l, m) go to the workspace and a second kernel joins the parts, always
// in the order of the keys.  Every CTA finds its share from the metadata by
// itself, in one block-wide sum: no plan, no counters, nothing to be cleared.
//
// One warp has the pages copied into a ring of stages by the TMA engine; four
// warps take 16 rows by the keys of a stage, or by a half or a quarter of them
// (mma.sync 16 x 8 x 16: the products are far from the bound, and at most half of
// a 128-row tcgen05 tile would be used).
//
// What it takes, in a graph: 256 sequences of 500 to 4000, 32 / 8 heads of 128 bf16, 392 us,
// 6.1 TB/s, 0.92 of the copy rate; two of 130000 and less, 16 / 2 heads, 50 us for 27; 32
// of 5 drafts, 20 / 4 heads of 96, 50 us for 24 (launched one by one 397, 54 and 54 to 57).  The
// first is 1.6 us a key tile and CTA, the memory's rate; the other two have 18 and 21 of
// them, and beside those a part that every call has: 6 us until the first product, the
// runs' ends, the join (7 to 17 us by itself with cold caches).
#include "ssu_paged.cuh"
#include "ssu_tcgen05.cuh"

namespace ssu {

namespace {

constexpr int kKeys = 64;             // keys of a stage
constexpr int kPanel = kKeys * 128;   // bytes of 64 elements of its keys
constexpr int kWarps = 4;             // consumers
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kCtas = 2;              // per SM

constexpr float kLift = 15.f;         // log2 by which fp16 weights are larger than the softmax's before its division

template <int DK, int MT>
struct Layout {
    static constexpr int kPanels = (DK + 63) / 64;
    static constexpr int kRows = 16 * MT;
    static constexpr int kStageBytes = 2 * kPanels * kPanel;
    static constexpr int kStages = DK == 64 ? 6 : 3;
    static constexpr int kQ = kStages * kStageBytes;                 // [kRows][64 kPanels], 16-byte pieces swapped by row
    static constexpr int kQRow = kPanels * 128;
    static constexpr int kSlice = 32 / MT;                           // columns joined at a time
    static constexpr int kJoin = kQ;                                 // [kWarps / MT][kRows][kSlice] fp32, once the queries are done with
    static constexpr int kJoinBytes = kWarps / MT * kRows * kSlice * 4;
    static constexpr int kML = kQ + (kRows * kQRow > kJoinBytes ? kRows * kQRow : kJoinBytes);  // [kWarps / MT][kRows][2]
    static constexpr int kBar = kML + kWarps / MT * kRows * 8;
    static constexpr int kMisc = kBar + 16 * kStages;
    static constexpr int kBytes = kMisc + 128;
    static constexpr int kPart = kRows * (DK + 2);                   // floats of a part in the workspace: o, l, m
    static_assert(kBytes <= (228 * 1024) / kCtas - 1024, "shared memory");  // (1 KB of an SM's goes with every CTA)
};

// What the second kernel has to know of a CTA's first run: the row tile that it
// continues (b < 0: none) and whether it is the tile's last.
struct Joint {
    int32_t b, g, tile, last;
};

__device__ __forceinline__ int row_tiles(const PagedParams &p, const Seq &s, int rows) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.share + rows - 1) / rows);
}

// A row tile's keys.
struct Range {
    int pos_lo, pos_hi;  // positions of its first and last token
    int lo, end;         // keys that any of its rows sees: [lo, end)
    int first, count;    // key tiles; one at least
};
__device__ __forceinline__ Range range_of(const AttendParams &p, const Seq &s, int tile, int rows) {
    Range r;
    const int64_t m0 = static_cast<int64_t>(tile) * rows, all = static_cast<int64_t>(s.n) * p.c.share;
    const int64_t m1 = min(m0 + rows, all) - 1;
    r.pos_lo = s.kv - s.n + static_cast<int>(m0 / p.c.share);
    r.pos_hi = s.kv - s.n + static_cast<int>(m1 / p.c.share);
    r.end = max(r.pos_hi + 1, 0);
    r.lo = p.window > 0 ? max(r.pos_lo - p.window + 1, 0) : 0;
    if (r.lo > r.end) r.lo = r.end;
    r.first = r.lo / kKeys;
    r.count = max((r.end + kKeys - 1) / kKeys - r.first, 1);
    return r;
}
// Key tiles of all row tiles of a sequence, for one head.
__device__ __forceinline__ int64_t tiles_of(const AttendParams &p, const Seq &s, int rows) {
    int64_t sum = 0;
    const int n = row_tiles(p.c, s, rows);
    for (int t = 0; t < n; ++t) sum += range_of(p, s, t, rows).count;
    return sum;
}

// A CTA's share: where it begins, and how many key tiles it has.
struct Share {
    int64_t left;
    int32_t b, g, tile, at;  // sequence, head, row tile, key tile of it
};

// The share's runs, one row tile after the other.
struct Walk {
    Share w;
    Seq s;
    int tiles;
    Range r;
    __device__ __forceinline__ void start(const AttendParams &p, const Share &share, int rows) {
        w = share;
        if (w.left <= 0) return;
        s = load_seq(p.c, w.b, false);
        tiles = row_tiles(p.c, s, rows);
        r = range_of(p, s, w.tile, rows);
    }
    __device__ __forceinline__ bool more() const { return w.left > 0; }
    // key tiles [at, at + run()) of the row tile
    __device__ __forceinline__ int run() const { return static_cast<int>(min(static_cast<int64_t>(r.count - w.at), w.left)); }
    __device__ __forceinline__ void next(const AttendParams &p, int rows) {
        w.left -= run();
        w.at = 0;
        if (w.left <= 0) return;
        if (++w.g == p.c.G) {
            w.g = 0;
            if (++w.tile >= tiles) {
                w.tile = 0;
                do {  // (the share ends within a sequence that has rows, unless the lengths changed meanwhile)
                    if (++w.b >= p.c.nseq) {
                        w.left = 0;
                        return;
                    }
                    s = load_seq(p.c, w.b, false);
                } while (s.n == 0);
                tiles = row_tiles(p.c, s, rows);
            }
            r = range_of(p, s, w.tile, rows);
        }
    }
};

// This CTA's share, by all of its threads; `sums` holds one number per warp.
__device__ __forceinline__ void find_share(const AttendParams &p, int rows, int64_t *sums, Share *out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t per = (p.c.nseq + kThreads - 1) / kThreads;
    const int64_t b0 = min(tid * per, p.c.nseq), b1 = min(b0 + per, p.c.nseq);
    int64_t mine = 0;
    for (int64_t b = b0; b < b1; ++b) mine += tiles_of(p, load_seq(p.c, b, blockIdx.x == 0), rows) * p.c.G;
    int64_t upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
    }
    if (lane == 31) sums[warp] = upto;
    if (tid == 0) out->left = 0;
    __syncthreads();
    int64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < kWarps + 1; ++w) {
        if (w == warp) before = total;
        total += sums[w];
    }
    const int64_t from = before + upto - mine;
    // no share is empty but those of the last CTAs, where there are fewer key tiles than CTAs
    const int64_t n = min(total, static_cast<int64_t>(gridDim.x)), c = blockIdx.x;
    const auto start = [&](int64_t i) { return total / n * i + total % n * i / n; };
    if (c >= n) return;
    const int64_t w0 = start(c), w1 = start(c + 1);
    if (w0 >= from && w0 < from + mine) {
        int64_t at = w0 - from;
        for (int64_t b = b0; b < b1; ++b) {
            const Seq s = load_seq(p.c, b, false);
            const int tiles = row_tiles(p.c, s, rows);
            for (int t = 0; t < tiles; ++t) {
                const int count = range_of(p, s, t, rows).count;
                const int64_t all = static_cast<int64_t>(count) * p.c.G;
                if (at < all) {
                    out->b = static_cast<int32_t>(b);
                    out->tile = t;
                    out->g = static_cast<int32_t>(at / count);
                    out->at = static_cast<int32_t>(at % count);
                    out->left = w1 - w0;
                    b = b1;
                    break;
                }
                at -= all;
            }
        }
    }
    __syncthreads();
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t saddr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_t(uint32_t saddr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, const uint32_t *b) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF) {
        return pack_bf16x2(a, b);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
template <bool BF>
__device__ __forceinline__ float value_of(unsigned short u) {
    return bits_to_float(u, BF ? kBF16 : kF16);
}
// Where element `dim` of key `row` lies in a stage's panels.
__device__ __forceinline__ uint32_t place(int row, int dim) {
    return (dim >> 6) * kPanel + row * 128 + ((((dim & 63) >> 3) ^ (row & 7)) * 16);
}

// What a row's outputs become: o / l, zeros where the row sees nothing.
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.6931471805599453f; }

// Four columns of one row's outputs.
template <bool BF>
__device__ __forceinline__ void store_out(const AttendParams &p, const Seq &s, int g, int64_t m, int dim, const float *o, int n) {
    if (dim >= p.c.D) return;
    const int64_t row = s.t0 + m / p.c.share;
    const int h = g * p.c.share + static_cast<int>(m % p.c.share);
    unsigned short *out = static_cast<unsigned short *>(p.c.out) + row * p.c.os[0] + h * p.c.os[1] + dim;
#pragma unroll
    for (int i = 0; i < 4; i += 2)
        if (i < n) *reinterpret_cast<uint32_t *>(out + i) = pack2<BF>(o[i], o[i + 1]);
}
__device__ __forceinline__ void store_lse(const AttendParams &p, const Seq &s, int g, int64_t m, float lse) {
    if (p.lse) p.lse[(s.t0 + m / p.c.share) * p.c.H + g * p.c.share + m % p.c.share] = lse;
}

// DK: the head size, rounded up to 64, 96 or 128; MT: row tiles of 16; BF: bf16.
template <int DK, int MT, bool BF>
__global__ void __launch_bounds__(kThreads, kCtas) attend_rows_kernel(const AttendParams p, const __grid_constant__ CacheMaps maps,
                                                                      int box, Joint *joints, float *parts) {
    using LY = Layout<DK, MT>;
    constexpr int R = LY::kRows;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + LY::kBar), *const empty = full + LY::kStages;
    Share *const share = reinterpret_cast<Share *>(smem + LY::kMisc);
    int *const abort_flag = reinterpret_cast<int *>(smem + LY::kMisc + 32), *const odd_flag = abort_flag + 1;
    int64_t *const sums = reinterpret_cast<int64_t *>(smem + LY::kMisc + 48);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        *abort_flag = 0;
        *odd_flag = 0;
        for (int i = 0; i < LY::kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], kWarps);
    }
    start_dependents();
    find_share(p, R, sums, share);  // (its barriers order the set-up too)
    Walk walk;
    walk.start(p, *share, R);
    if (tid == 0) {
        Joint j{-1, 0, 0, 0};
        if (walk.more() && walk.w.at > 0) j = {walk.w.b, walk.w.g, walk.w.tile, walk.w.at + walk.run() == walk.r.count};
        joints[blockIdx.x] = j;
    }
    bool ok = true;
    if (warp == kWarps) {
        // ---------------- copies ----------------
        const PageCopier<kKeys, LY::kPanels> pages(p.c, box);
        int it = 0;
        const auto look_up = [&](int at) { return pages.look_up(walk.w.b, walk.r.first + at, walk.r.lo, walk.r.end); };
        int page = walk.more() ? look_up(walk.w.at) : 0;
        while (ok && walk.more()) {
            const int from = walk.w.at, to = from + walk.run(), g = walk.w.g;
            for (int i = from; i < to; ++i, ++it) {
                const int s = it % LY::kStages;
                const auto here = pages.find(page, walk.r.first + i, walk.r.lo, walk.r.end);
                if (i + 1 < to) {
                    page = look_up(i + 1);
                } else {
                    walk.next(p, R);
                    if (walk.more()) page = look_up(walk.w.at);
                }
                if (it >= LY::kStages) ok = mbar_wait_bounded(&empty[s], (it / LY::kStages - 1) & 1);
                ok = __all_sync(0xffffffffu, ok && !*reinterpret_cast<volatile int *>(abort_flag));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect(&full[s], 2 * here.bytes);
                __syncwarp();
                const uint32_t dst = smem_addr(smem + s * LY::kStageBytes);
                pages.copy(here, maps.k, g, dst, &full[s]);
                pages.copy(here, maps.v, g, dst + LY::kPanels * kPanel, &full[s]);
            }
        }
        if (!ok) {
            if (lane == 0) flag(p.c.status, kDevTimeout);
            *abort_flag = 1;
        }
        // what was asked for has landed before the CTA retires
        if (lane == 0)
            for (int k = max(it - LY::kStages, 0); k < it; ++k) mbar_wait_bounded(&full[k % LY::kStages], (k / LY::kStages) & 1);
        __syncwarp();
        return;
    }

    // ---------------- consumers ----------------
    const uint32_t s0 = smem_addr(smem);
    float *const join = reinterpret_cast<float *>(smem + LY::kJoin);
    float2 *const ml = reinterpret_cast<float2 *>(smem + LY::kML);
    const float scale = p.scale * 1.4426950408889634f;
    int it = 0;
    bool first_run = true;
    for (; ok && walk.more(); walk.next(p, R), first_run = false) {
        const Seq s = walk.s;
        const Range r = walk.r;
        const int g = walk.w.g, from = walk.w.at, to = from + walk.run();
        const int64_t m0 = static_cast<int64_t>(walk.w.tile) * R;
        const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(s.n) * p.c.share - m0));
        // the queries
        for (int i = tid; i < R * DK / 8; i += 32 * kWarps) {
            const int row = i / (DK / 8), piece = i % (DK / 8);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (row < rows && 8 * piece < p.c.D) {
                const int64_t m = m0 + row;
                v = __ldg(reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(p.c.q) + (s.t0 + m / p.c.share) * p.c.qs[0] +
                                                          (g * p.c.share + m % p.c.share) * p.c.qs[1] + 8 * piece));
            }
            *reinterpret_cast<uint4 *>(smem + LY::kQ + row * LY::kQRow + ((piece ^ (row & 7)) * 16)) = v;
        }
        named_barrier(1, 32 * kWarps);
        // this warp's 16 rows, and its keys of a tile: 16 of every MT x 16 that it shares with the warps of the other rows
        const int row0 = 16 * (warp % MT), keys0 = 16 * MT * (warp / MT);
        uint32_t q[DK / 16][4];
#pragma unroll
        for (int k = 0; k < DK / 16; ++k) {
            const int row = row0 + (lane & 15), piece = 2 * k + (lane >> 4);
            ldmatrix_x4(s0 + LY::kQ + row * LY::kQRow + ((piece ^ (row & 7)) * 16), q[k]);
        }
        // this thread's rows: lane / 4 and lane / 4 + 8 of those
        float mx[2], sum[2], o[DK / 8][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) mx[h] = -INFINITY, sum[h] = 0.f;
#pragma unroll
        for (int n = 0; n < DK / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;

        bool ended = false;
        for (int i = from; i < to; ++i, ++it) {
            const int st = it % LY::kStages;
            ok = mbar_wait_bounded(&full[st], (it / LY::kStages) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t sk = s0 + st * LY::kStageBytes, sv = sk + LY::kPanels * kPanel;
            const int key0 = (r.first + i) * kKeys;
            // all rows see all of the tile?
            const bool masked = key0 + kKeys > r.pos_lo + 1 || (p.window > 0 && key0 < r.pos_hi + 1 - p.window);
            if (masked) {
                // Values that some row does not see must not reach it by a zero
                // of P: what no row sees becomes zeros, and so do infinities
                // and NaN, which are added to the rows that see them at the end.
                // (A warp its own keys, or its part of those it shares.)
                unsigned char *const values = smem + st * LY::kStageBytes + LY::kPanels * kPanel;
                const bool partly = r.pos_lo != r.pos_hi;
                bool odd = false;
                for (int e = lane; e < 16 * (DK / 8); e += 32) {
                    const int row = 16 * warp + e / (DK / 8), key = key0 + row;
                    uint4 *const v = reinterpret_cast<uint4 *>(values + place(row, 8 * (e % (DK / 8))));
                    if (key >= r.end || key < r.lo) {
                        *v = make_uint4(0u, 0u, 0u, 0u);
                    } else if (partly && any_odd<BF>(*v)) {
                        odd = true;
                        *v = without_odd<BF>(*v);
                    }
                }
                if (odd) *odd_flag = 1;
                fence_proxy_async_smem();  // before the stage's next copy
                if (MT == 1) {
                    __syncwarp();
                } else if (barrier_or(1, 32 * kWarps, false)) {  // a warp whose wait gave up is at the run's end: this was it
                    ok = false, ended = true;
                    break;
                }
            }
            constexpr int kSub = MT == 1 ? 1 : 2;  // 16 keys at a time, or 32
#pragma unroll 1
            for (int sub = 0; sub < MT; sub += kSub) {
                const int mine = keys0 + 16 * sub;
                float x[2 * kSub][4];
#pragma unroll
                for (int n = 0; n < 2 * kSub; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[n][j] = 0.f;
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
#pragma unroll
                    for (int n = 0; n < kSub; ++n) {
                        uint32_t b[4];
                        ldmatrix_x4(sk + place(mine + 16 * n + (lane & 7) + ((lane >> 4) << 3), 16 * k + ((lane >> 3) & 1) * 8), b);
                        mma16816<BF>(x[2 * n], q[k], b);
                        mma16816<BF>(x[2 * n + 1], q[k], b + 2);
                    }
                // P and the running maximum and sum
                uint32_t pa[kSub][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float e[4 * kSub];  // keys 8 (j / 2) + 2 (lane % 4) + j % 2 of the row
#pragma unroll
                    for (int j = 0; j < 4 * kSub; ++j) e[j] = __fmul_rn(x[j / 2][2 * h + j % 2], scale);  // (rounded, as the maximum is: none is above it)
                    if (masked) {
                        // (the row's position, found here: kept it would cost registers on every tile)
                        const int row = min(row0 + 8 * h + lane / 4, rows - 1);
                        const int pos = s.kv - s.n + static_cast<int>((m0 + row) / p.c.share);
#pragma unroll
                        for (int j = 0; j < 4 * kSub; ++j) {
                            const int key = key0 + mine + 8 * (j >> 1) + 2 * (lane & 3) + (j & 1);
                            if (key > pos || (p.window > 0 && key <= pos - p.window)) e[j] = -INFINITY;
                        }
                    }
                    float top = BF ? mx[h] : -INFINITY;
#pragma unroll
                    for (int j = 0; j < 4 * kSub; ++j) top = fmaxf(top, e[j]);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // (where fp32 has no halves left the difference might be rounded up, past fp16's range)
                    if constexpr (!BF) top = fmaxf(mx[h], fabsf(top) < 8388608.f ? top - kLift : top);
                    const float base = top == -INFINITY ? 0.f : top, back = ex2(mx[h] - base);
                    mx[h] = top;
                    float add = 0.f;
#pragma unroll
                    for (int j = 0; j < 4 * kSub; ++j) {
                        e[j] = ex2(e[j] - base);
                        add += e[j];
                    }
                    sum[h] = sum[h] * back + add;
                    if (back != 1.f)
#pragma unroll
                        for (int n = 0; n < DK / 8; ++n) o[n][2 * h] *= back, o[n][2 * h + 1] *= back;
#pragma unroll
                    for (int n = 0; n < kSub; ++n) pa[n][h] = pack2<BF>(e[4 * n], e[4 * n + 1]), pa[n][2 + h] = pack2<BF>(e[4 * n + 2], e[4 * n + 3]);
                }
#pragma unroll
                for (int n = 0; n < DK / 16; ++n)
#pragma unroll
                    for (int k = 0; k < kSub; ++k) {
                        uint32_t b[4];
                        ldmatrix_x4_t(sv + place(mine + 16 * k + (lane & 15), 16 * n + ((lane >> 4) << 3)), b);
                        mma16816<BF>(o[2 * n], pa[k], b);
                        mma16816<BF>(o[2 * n + 1], pa[k], b + 2);
                    }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }
        if (!ended) ok = !barrier_or(1, 32 * kWarps, !ok);
        if (!ok) break;

        // ---------------- the warps' parts joined ----------------
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float t = sum[h];
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            if ((lane & 3) == 0) ml[warp / MT * R + row0 + 8 * h + lane / 4] = make_float2(mx[h], t);
        }
        named_barrier(1, 32 * kWarps);
        constexpr int kSets = kWarps / MT;  // warps that share a row
        const auto top_of = [&](int row) {
            float m = ml[row].x;
#pragma unroll
            for (int w = 1; w < kSets; ++w) m = fmaxf(m, ml[w * R + row].x);
            return m;
        };
        const bool whole = from == 0 && to == r.count, odd = *odd_flag != 0;
        // (the part of a cut run: a continuation is its CTA's first run, another its last)
        float *const part = parts + (2 * static_cast<int64_t>(blockIdx.x) + (from > 0 ? 0 : 1)) * LY::kPart;
        float down[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float m = top_of(row0 + 8 * h + lane / 4);
            down[h] = mx[h] == -INFINITY ? 0.f : ex2(mx[h] - m);
        }
        // a thread takes kWide columns of one row of each slice
        constexpr int kWide = R * LY::kSlice / (32 * kWarps), kAcross = LY::kSlice / kWide;
        static_assert(kWide == 4, "a thread's columns");
        const int row = tid / kAcross, col = tid % kAcross * kWide;
        const float m = top_of(row);
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kSets; ++w) {
            const float2 f = ml[w * R + row];
            l += f.y * (f.x == -INFINITY ? 0.f : ex2(f.x - m));  // (a sum without a maximum is 0 or NaN)
        }
        const int pos = s.kv - s.n + static_cast<int>((m0 + min(row, rows - 1)) / p.c.share);
        const float inv = 1.f / l;
#pragma unroll
        for (int c = 0; c < DK; c += LY::kSlice) {
#pragma unroll
            for (int n = c / 8; n < (c + LY::kSlice) / 8; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(&join[(warp / MT * R + row0 + 8 * h + lane / 4) * LY::kSlice + 8 * n - c + 2 * (lane & 3)]) =
                        make_float2(o[n][2 * h] * down[h], o[n][2 * h + 1] * down[h]);
            named_barrier(1, 32 * kWarps);
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kSets; ++w) {
                const float4 f = *reinterpret_cast<const float4 *>(&join[(w * R + row) * LY::kSlice + col]);
                v[0] += f.x, v[1] += f.y, v[2] += f.z, v[3] += f.w;
            }
            named_barrier(1, 32 * kWarps);
            if (__builtin_expect(odd, 0) && row < rows && c + col < p.c.D) {
                // infinities and NaN that were left out, of the keys this row sees in the run
                const int k0 = max((r.first + from) * kKeys, p.window > 0 ? pos + 1 - p.window : 0);
                const int k1 = min((r.first + to) * kKeys, pos + 1);
                for (int key = max(k0, 0); key < k1; ++key) {
                    const int tile0 = key / kKeys * kKeys;
                    if (!(tile0 + kKeys > r.pos_lo + 1 || (p.window > 0 && tile0 < r.pos_hi + 1 - p.window))) continue;
                    const int64_t page = page_of(p.c, walk.w.b, key);
                    if (page < 0) continue;
                    const unsigned short *at = static_cast<const unsigned short *>(p.c.v_cache) + page * p.c.vs[0] +
                                               (key % p.c.page) * p.c.vs[1] + g * p.c.vs[2] + c + col;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float f = value_of<BF>(__ldg(at + k));
                        if (!(fabsf(f) <= 3.402823466e38f)) v[k] += f;
                    }
                }
            }
            if (whole) {
                if (row < rows) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = pos < 0 ? 0.f : v[k] * inv;
                    store_out<BF>(p, s, g, m0 + row, c + col, v, 4);
                }
            } else {
                *reinterpret_cast<float4 *>(&part[row * DK + c + col]) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        if (tid % kAcross == 0) {
            if (!whole) part[R * DK + row] = l, part[R * DK + R + row] = m;
            else if (row < rows) store_lse(p, s, g, m0 + row, pos < 0 ? -INFINITY : lse_of(m, l));
        }
        named_barrier(1, 32 * kWarps);
        if (odd && tid == 0) *odd_flag = 0;  // (read again after the next run's first barrier)
    }
    if (!ok) {
        if (lane == 0) flag(p.c.status, kDevTimeout);
        *abort_flag = 1;
    }
}

// The parts of the row tile that CTA c's share begins within, if it is the first
// that does: the end of share c - 1, the beginnings of c, c + 1, ...  Four warps
// take a row, each a quarter of its parts, a lane four columns; what they sum is
// added in the order of the keys' quarters.
constexpr int kJoinRows = 4, kJoinSlices = 4;
template <int DK, int MT, bool BF>
__global__ void __launch_bounds__(32 * kJoinRows * kJoinSlices) attend_join_kernel(const AttendParams p, int ctas, const Joint *joints,
                                                                                   const float *parts) {
    using LY = Layout<DK, MT>;
    constexpr int R = LY::kRows;
    __shared__ float4 sums[kJoinRows][kJoinSlices][32];
    __shared__ float ls[kJoinRows][kJoinSlices];
    const int c = blockIdx.x + 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_prior();
    const Joint j = joints[c];
    if (j.b < 0) return;
    const Joint before = joints[c - 1];
    // (share c - 1 lies within the same tile: an earlier CTA joins it)
    if (before.b == j.b && before.g == j.g && before.tile == j.tile && !before.last) return;
    int last = c;
    for (;; last += 32) {
        const uint32_t ends = __ballot_sync(0xffffffffu, last + lane >= ctas - 1 || joints[last + lane].last);
        if (ends != 0) {
            last += __ffs(ends) - 1;
            break;
        }
    }
    const Seq s = load_seq(p.c, j.b, false);
    const int64_t m0 = static_cast<int64_t>(j.tile) * R;
    const int rows = static_cast<int>(min(static_cast<int64_t>(R), static_cast<int64_t>(s.n) * p.c.share - m0));
    const int row = blockIdx.y * kJoinRows + warp / kJoinSlices, slice = warp % kJoinSlices;
    const auto part = [&](int i) { return parts + (i < c ? 2 * static_cast<int64_t>(c - 1) + 1 : 2 * static_cast<int64_t>(i)) * LY::kPart; };
    const bool mine = 4 * lane < DK;
    float m = -INFINITY;
    if (row < rows) {
        for (int i = c - 1 + lane; i <= last; i += 32) m = fmaxf(m, part(i)[R * DK + R + row]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        const int n = last - c + 2, i0 = c - 1 + n * slice / kJoinSlices, i1 = c - 1 + n * (slice + 1) / kJoinSlices;
        float l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
            const float *q = part(i);
            const float top = q[R * DK + R + row], f = top == -INFINITY ? 0.f : ex2(top - m);
            l += q[R * DK + row] * f;
            if (mine) {
                const float4 o = *reinterpret_cast<const float4 *>(&q[row * DK + 4 * lane]);
                v.x += o.x * f, v.y += o.y * f, v.z += o.z * f, v.w += o.w * f;
            }
        }
        sums[warp / kJoinSlices][slice][lane] = v;
        if (lane == 0) ls[warp / kJoinSlices][slice] = l;
    }
    __syncthreads();
    if (row >= rows || slice != 0) return;
    float l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kJoinSlices; ++k) {
        const float4 o = sums[warp / kJoinSlices][k][lane];
        l += ls[warp / kJoinSlices][k];
        v[0] += o.x, v[1] += o.y, v[2] += o.z, v[3] += o.w;
    }
    const int pos = s.kv - s.n + static_cast<int>((m0 + row) / p.c.share);
    const float inv = 1.f / l;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pos < 0 ? 0.f : v[k] * inv;
    if (mine) store_out<BF>(p, s, j.g, m0 + row, 4 * lane, v, 4);
    if (lane == 0) store_lse(p, s, j.g, m0 + row, pos < 0 ? -INFINITY : lse_of(m, l));
}

int rows_grid() {
    // not the device's count: the workspace's size and the launch have to agree on it (with fewer SMs
    // some take a second CTA's share)
    constexpr int kSms = 152;
    return kCtas * kSms;
}

template <int DK, int MT, bool BF>
cudaError_t launch_t(const AttendParams &p, void *workspace, cudaStream_t stream) {
    using LY = Layout<DK, MT>;
    // Before the maps: their encoder is a driver call and refuses a host thread
    // that has no context yet, which this one gives it.
    cudaError_t e = cudaFuncSetAttribute(attend_rows_kernel<DK, MT, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, LY::kBytes);
    if (e != cudaSuccess) return e;
    CacheMaps maps;
    if (!encode_cache(&maps, p.c, kKeys)) return cudaErrorInvalidValue;
    const int grid = rows_grid();
    Joint *joints = static_cast<Joint *>(workspace);
    float *parts = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + (grid * sizeof(Joint) + 255) / 256 * 256);
    attend_rows_kernel<DK, MT, BF><<<grid, kThreads, LY::kBytes, stream>>>(p, maps, least_box(p.c, kKeys), joints, parts);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_after(attend_join_kernel<DK, MT, BF>, dim3(grid - 1, LY::kRows / kJoinRows), 32 * kJoinRows * kJoinSlices, 0, stream, p, grid,
                        joints, parts);
}
template <int DK, int MT>
cudaError_t launch_m(const AttendParams &p, void *workspace, cudaStream_t stream) {
    return p.c.io_dtype == kBF16 ? launch_t<DK, MT, true>(p, workspace, stream) : launch_t<DK, MT, false>(p, workspace, stream);
}

template <int DK>
cudaError_t launch_d(const AttendParams &p, int kind, void *workspace, cudaStream_t stream) {
    if (kind == kAttendRows16) return launch_m<DK, 1>(p, workspace, stream);
    if (kind == kAttendRows32) return launch_m<DK, 2>(p, workspace, stream);
    return launch_m<DK, 4>(p, workspace, stream);
}

}  // namespace

uint64_t attend_rows_workspace(int kind, int D) {
    const uint64_t rows = kind == kAttendRows16 ? 16 : kind == kAttendRows32 ? 32 : 64, dk = D <= 64 ? 64 : D <= 96 ? 96 : 128;
    return (rows_grid() * sizeof(Joint) + 255) / 256 * 256 + 2 * rows_grid() * rows * (dk + 2) * sizeof(float);
}

cudaError_t launch_attend_rows(const AttendParams &p, int kind, void *workspace, cudaStream_t stream) {
    if (p.c.D <= 64) return launch_d<64>(p, kind, workspace, stream);
    if (p.c.D <= 96) return launch_d<96>(p, kind, workspace, stream);
    return launch_d<128>(p, kind, workspace, stream);
}

}  // namespace ssu
