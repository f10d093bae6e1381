// ssu_paged_tiles.cu -- attention over the paged cache on the 5th-generation
// tensor cores: chunks of prompts, and batches that hold some.
//
// A work unit is up to 2 x 128 query rows of one sequence and key/value head --
// tile A and tile B, each floor(128 / share) tokens by `share` heads, the head
// fastest -- over the 128-key tiles that its rows see.  One pass over the keys
// with a running reference m and sum l, in units of log2:
//     x_j = scale log2(e) q . k_j,   P_j = 2^(x_j - m),   l += sum P_j,   O += P V
// and out = O / l, lse = (m + log2 l) ln 2.  m is the row's maximum when it was last
// moved (fp16: less 7); it moves when P would pass 2^8 (fp16: 2^15), so that O, in
// tensor memory, is rarely rescaled (that is inside both io types,
// and l and O are fp32; scores are scaled and their difference taken in one rounding,
// in two where |m| is so large that this would not keep P there).  P is rounded once to the io type, as its product's operand.
//
// A plan kernel checks the metadata, lists the units and, where they are too few
// or too uneven for the GPU, cuts their keys into parts; the main kernel's CTAs
// take the list in turn.  Parts leave (O, l, m) in the workspace, where a third
// kernel joins them in the order of the keys.
//
// Two products a key tile and query tile, fp32 accumulators in tensor memory:
//     S = Q K^T  (both from shared memory, as copied),  O += P V  (P where S was)
// Warps, in groups of four:
//   0-3, 4-7  (thread = row of tile A, B) S -> P, O rescaled;
//   8         issues the products;   9  finds the units and copies pages;
//   10-11     look through the values of partly visible tiles (below);
//   12-15     store the outputs.
//
// What it takes: 32768 tokens in 16 prompts, 32 / 8 heads of 128 bf16, 562 us in a graph, 1250
// TFLOP/s, 0.65 of the measured product rate (571 us launched one by one); 2432 tokens
// behind 65536, 16 / 4 heads, 751 us, 1770 TFLOP/s, the measured sustained rate.  A key tile takes 2800 cycles
// for both row tiles, of which the products alone would be 2048: S reads both its
// operands from shared memory at the pipe's whole rate while copies are written, and
// a tile's chain -- scores, 1450 cycles of softmax, P V and the next scores -- is as
// long.  A unit's turnover takes about 5000 more.
#include <type_traits>

#include "ssu_paged.cuh"
#include "ssu_tcgen05.cuh"

namespace ssu {

namespace {

constexpr int kRows = 128;     // rows of a query tile
constexpr int kKeys = 128;     // keys of a tile
constexpr int kPanel = 16384;  // 128 rows of 128 bytes
constexpr int kThreads = 512;
// The reference moves to the maximum less kLift when that is more than kMost above it.
// For fp16 P is between 2^7 and 2^15 where it is largest, so that it is rounded by half a step down
// to 2^-21 of the largest weight and by 2^-32 of it below, 2^21 tokens of which come to half a step
// of the whole: with 0 and 8 as for bf16, the tokens of a long context beside one that takes nearly
// all the weight, 2^-25 of it each, were nothing.  (With 11 and 15 O is rescaled more often: 43
// sequences of single tokens and chunks 257 us, 246 so.)
template <bool BF>
constexpr float kLift = BF ? 0.f : 7.f;
template <bool BF>
constexpr float kMost = BF ? 8.f : 15.f;
// References from here on are too coarse for exponents formed in one rounding, scale s - m: the
// reference is a rounded product, half a step of which is 2^-4 here and whole units of log2 soon.
constexpr float kCoarse = 1048576.f;

// A part of a unit's keys, as planned.
struct Piece {
    int64_t row0;         // first row of the sequence's new tokens
    int32_t b, n, kv;     // sequence, its new tokens, its tokens in the cache
    int32_t pair;         // tokens [pair, pair + 1) * 2 * (128 / share) of it
    int32_t first, last;  // key tiles
    int32_t part, parts;  // of the unit's parts, which
    int32_t slot;         // the first part's place in the workspace (where parts > 1)
};
struct PlanHead {
    int32_t pieces, cuts, next;  // number of pieces, of units that are cut; the next piece to be taken
};
struct Plan {
    PlanHead *head;
    Piece *units, *pieces;  // whole units; parts, where some are cut
    int32_t *cuts;          // the first part of every unit that is cut
    float *parts;           // [slots][G][2][kRows][DK + 2]
    int32_t max_units, max_slots;  // what there is room for: units; parts of cut units (a head)
};

// What the groups need to know of a piece.
struct Work {
    int64_t row[2];            // first row of tile A, B
    int32_t b, g;
    int32_t toks[2], pos[2];   // tokens, position of the first
    int32_t from[2], to[2];    // key tiles
    int32_t first, last;       // of either; last < 0: no more work
    int32_t part, parts, slot;
};

__device__ __forceinline__ int tile_tokens(const PagedParams &p) { return kRows / p.share; }

// Key tiles that tokens at positions [pos, pos + toks) see.
__device__ __forceinline__ void key_tiles(const AttendParams &p, int pos, int toks, int &from, int &to) {
    const int end = max(pos + toks, 0);
    const int lo = p.window > 0 ? max(pos + 1 - p.window, 0) : 0;
    from = lo / kKeys;
    to = toks > 0 && end > lo ? (end + kKeys - 1) / kKeys : from;
}
// Does every row of the tile see all of key tile j?
__device__ __forceinline__ bool sees_all(int window, int pos, int toks, int j) {
    return (j + 1) * kKeys <= pos + 1 && (window == 0 || j * kKeys >= pos + toks - window);
}
__device__ __forceinline__ bool partly_seen(const Work &w, int window, int j) {
    bool some = false;
#pragma unroll
    for (int x = 0; x < 2; ++x)
        some = some || (j >= w.from[x] && j < w.to[x] && !sees_all(window, w.pos[x], w.toks[x], j));
    return some;
}

// ---------------------------------------------------------------------------
// The plan: one CTA.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 256;
constexpr int kMaxParts = 64;

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < kPlanThreads / 32 ? red[lane] : 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}
// Sum of the threads before this one; `total` of all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *red, int64_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t upto = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += o;
    }
    __syncthreads();
    if (lane == 31) red[warp] = upto;
    __syncthreads();
    int64_t w = lane < kPlanThreads / 32 ? red[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, w, off);
        if (lane >= off) w += o;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return upto - v + (warp > 0 ? before : 0);
}
// Key tiles of a pair of tiles.
__device__ __forceinline__ void pair_tiles(const AttendParams &p, const Seq &s, int pair, int &first, int &last) {
    const int tt = tile_tokens(p.c), t0 = pair * 2 * tt, pos = s.kv - s.n + t0;
    int f[2], l[2];
    key_tiles(p, pos, min(tt, s.n - t0), f[0], l[0]);
    key_tiles(p, pos + tt, max(min(tt, s.n - t0 - tt), 0), f[1], l[1]);
    first = f[0], last = l[0];
    if (l[1] > f[1]) {
        if (last == first) first = f[1];
        last = l[1];
    }
}

// How a unit of c key tiles is cut: `large` parts of `even` tiles, and the rest in
// parts of about `fine`, at most kMaxParts in all.
struct Cut {
    int large, parts;
};
__device__ __forceinline__ Cut cut_of(int c, int even, int fine, bool whole) {
    Cut k{0, 1};
    if (whole) return k;
    k.large = c / even;
    if (k.large >= kMaxParts) {  // (alike, then)
        k.large = 0;
        k.parts = kMaxParts;
        return k;
    }
    const int rest = c - k.large * even;
    k.parts = max(k.large + min((rest + fine - 1) / fine, kMaxParts - k.large), 1);
    return k;
}
// Key tiles [from, to) of its part i.
__device__ __forceinline__ void part_of(const Cut &k, int c, int even, int i, int &from, int &to) {
    const int large = min(k.large, k.parts);
    if (i < large) {
        from = i * even;
        to = i + 1 == k.parts ? c : from + even;
        return;
    }
    const int start = large * even, rest = c - start, n = k.parts - large, j = i - large;
    from = start + static_cast<int>(static_cast<int64_t>(rest) * j / n);
    to = start + static_cast<int>(static_cast<int64_t>(rest) * (j + 1) / n);
}

__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const AttendParams p, const Plan plan, int ctas) {
    start_dependents();
    __shared__ int64_t red64[32];
    __shared__ int bounds[kPlanThreads];
    const int tid = threadIdx.x, tt2 = 2 * tile_tokens(p.c);
    const auto pairs_of = [&](const Seq &s) { return (s.n + tt2 - 1) / tt2; };
    // The units, in the order of the sequences, the last tokens of each first.
    int64_t sum = 0;  // all key tiles, and one a unit
    int units = 0;
    for (int64_t b0 = 0; b0 < p.c.nseq; b0 += kPlanThreads) {
        Seq s{0, 0, 0};
        if (b0 + tid < p.c.nseq) s = load_seq(p.c, b0 + tid, true);
        // (where sequences overlap there may be more units than there is room for, or than 32 bits count: those stay away)
        int64_t wanted;
        const int room = plan.max_units - units;
        bounds[tid] = static_cast<int>(min(block_scan(pairs_of(s), red64, wanted), static_cast<int64_t>(room)));
        const int total = static_cast<int>(min(wanted, static_cast<int64_t>(room)));
        __syncthreads();
        for (int i = tid; i < total; i += kPlanThreads) {
            int lo = 0, hi = kPlanThreads;  // the sequence: bounds[lo] <= i, the last such
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (bounds[mid] <= i) lo = mid;
                else hi = mid;
            }
            const Seq q = load_seq(p.c, b0 + lo, false);
            Piece u{};
            u.row0 = q.t0, u.b = static_cast<int32_t>(b0 + lo), u.n = q.n, u.kv = q.kv;
            u.pair = pairs_of(q) - 1 - (i - bounds[lo]);
            u.parts = 1;
            pair_tiles(p, q, u.pair, u.first, u.last);
            plan.units[units + i] = u;
            sum += u.last - u.first + 1;
        }
        units += total;
        __syncthreads();
    }
    sum = block_sum(sum, red64) * p.c.G;

    // What is cut, with the even share of a CTA, `even`: a unit that is much longer
    // than that, into parts of it and a rest; and, where the CTAs take the list in
    // less than six rounds and the last one leaves many of them idle, that round's
    // units.  The rests and those are cut finely.
    const int64_t n = static_cast<int64_t>(units) * p.c.G, rounds = n / ctas, left = n - rounds * ctas;
    const int64_t even64 = max((sum + ctas - 1) / ctas, static_cast<int64_t>(8));
    const int even = static_cast<int>(min(even64, static_cast<int64_t>(1 << 30)));
    const int64_t tail = rounds >= 6 || 20 * left >= 17 * ctas || (left == 0 && rounds > 0) ? units : (rounds * ctas + p.c.G - 1) / p.c.G;
    int fine = max(even / 8, 4);
    const auto cut_unit = [&](int u) {
        const int c = plan.units[u].last - plan.units[u].first;
        return cut_of(c, even, fine, u < tail && c <= even + even / 8);
    };
    bool cut_any = units > 0 && plan.max_slots > 1;
    for (int turn = 0; cut_any; ++turn) {
        int64_t cut = 0;
        for (int u = tid; u < units; u += kPlanThreads) {
            const int parts = cut_unit(u).parts;
            cut += parts > 1 ? parts : 0;
        }
        cut = block_sum(cut, red64);
        if (cut == 0 || (turn == 4 && cut > plan.max_slots)) cut_any = false;
        else if (cut <= plan.max_slots) break;
        else fine *= 2;
    }
    if (!cut_any) {
        if (tid == 0) plan.head->pieces = units, plan.head->cuts = 0, plan.head->next = ctas;
        return;
    }
    // The pieces: all first parts, all second ones, ... so that CTAs that are at
    // work at the same time read the same keys.  (Among those the units come in any
    // order, which nothing but the time depends on.)
    __shared__ int next_piece[kMaxParts + 1], next_slot, next_cut;
    if (tid <= kMaxParts) next_piece[tid] = 0;
    if (tid == 0) next_slot = next_cut = 0;
    __syncthreads();
    for (int u = tid; u < units; u += kPlanThreads) {
        const int parts = cut_unit(u).parts;
        for (int i = 0; i < parts; ++i) atomicAdd(&next_piece[i + 1], 1);
    }
    __syncthreads();
    if (tid == 0)
        for (int i = 0; i < kMaxParts; ++i) next_piece[i + 1] += next_piece[i];
    __syncthreads();
    const int pieces = next_piece[kMaxParts];
    __syncthreads();
    for (int u = tid; u < units; u += kPlanThreads) {
        const Cut k = cut_unit(u);
        Piece q = plan.units[u];
        const int first = q.first, c = q.last - q.first, slot = k.parts > 1 ? atomicAdd(&next_slot, k.parts) : 0;
        for (int i = 0; i < k.parts; ++i) {
            int from, to;
            part_of(k, c, even, i, from, to);
            q.first = first + from, q.last = first + to;
            q.part = i, q.parts = k.parts, q.slot = slot;
            const int at = atomicAdd(&next_piece[i], 1);
            plan.pieces[at] = q;
            if (i == 0 && k.parts > 1) plan.cuts[atomicAdd(&next_cut, 1)] = at;
        }
    }
    __syncthreads();
    if (tid == 0) plan.head->pieces = pieces, plan.head->cuts = next_cut, plan.head->next = ctas;
}

// ---------------------------------------------------------------------------
// The attention.
// ---------------------------------------------------------------------------
constexpr int kAhead = 4;  // pieces of work announced ahead of the slowest warp
enum : int {
    kQFull0, kQFull1, kQFree0, kQFree1,      // a tile's queries have landed, are done with
    kUnitFull0, kUnitFree0 = kUnitFull0 + kAhead, kUnitEnd = kUnitFree0 + kAhead,  // pieces of work
    kSFull0 = kUnitEnd, kSFull1,             // scores of tile A, B are there
    kPFull0, kPFull1,                        // ... and have become P
    kOFull0, kOFull1,                        // P has been added to O
    kORead0, kORead1,                        // a piece's O has been read
    kStat0, kStat1, kStatFree0, kStatFree1,  // a piece's sums and references are there, have been read
    kFinal,
    kRing,                                   // a buffer is full; then: is empty; then: its values are looked through
};
constexpr uint32_t kColS = 0, kColO = 256;   // tensor memory: S (then P) of A, B; O of A, B
constexpr int kReaders = 15;                 // warps that read a piece of work
// Pieces of work kept: one is written when every warp has begun the one kAhead
// before it, and a warp looks at the one that it is at and, the products, at the next.
constexpr int kWorks = 8;
static_assert(kWorks >= kAhead + 2, "pieces of work");

template <int DK>
struct Layout {
    static constexpr int kPanels = DK / 64;
    static constexpr int kTile = kPanels * kPanel;        // 128 queries, keys or values
    static constexpr int kBufs = DK == 64 ? 10 : 5;
    static constexpr int kBuf = 2 * kTile;                // after the queries of A and B
    static constexpr int kBars = kBuf + kBufs * kTile;
    static constexpr int kWork = kBars + 8 * (kRing + 3 * kBufs);
    static constexpr int kMisc = (kWork + kWorks * static_cast<int>(sizeof(Work)) + 15) / 16 * 16;  // tensor-memory address, abort; odd[kWorks][2]
    static constexpr int kStat = kMisc + 32;              // [2][kRows] sum, reference
    static constexpr int kBytes = kStat + 2 * kRows * 8;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

enum : int { kWideOut = 1 };  // the rows of out lie on 32-byte boundaries
struct Maps {
    CUtensorMap q;
    CacheMaps cache;
};

template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// A wait, bounded like every other, of warps that mostly wait: asleep for up to
// 20 us at a time unless the phase completes.  (Polling, 32768 tokens in 16 prompts
// took 570 us where they take 552.)  Some wait for as long as a piece takes: `limit` is
// the call's (waits_of).
__device__ __forceinline__ bool sleep_on(uint64_t *bar, uint32_t parity, long long limit) {
    const long long t0 = clock64();
    for (uint32_t i = 0; i < (1u << 26); ++i) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
        if (clock64() - t0 > limit) break;
    }
    return false;
}
// The longest sequence that the block table has room for.
int64_t room_of(const PagedParams &p) { return p.table_width < kPagedMaxLen / p.page ? p.table_width * p.page : kPagedMaxLen; }
// Cycles after which a wait gives up: what is enough for a copy or a product, and five times what
// the key tiles of the longest sequence that the table has room for take one CTA, as they may be
// one piece's.  (Waits that start anew while tiles are copied need no length: 592 us of those prompts' 560.)
long long waits_of(const PagedParams &p) { return kWaitCycles + room_of(p) / kKeys * 16384; }

// A number that is known when this is compiled.
template <int N>
struct Known {
    static constexpr int value = N;
    __device__ __forceinline__ constexpr operator int() const { return N; }
};

// Two floats at a time.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float v;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(v) : "f"(a), "f"(b), "f"(c));
    return v;
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

__device__ __forceinline__ float lse_of(float ref, float l) {
    return ((ref == -INFINITY ? 0.f : ref) + log2f(l)) * 0.6931471805599453f;
}
// The place of a part of tile x: O as [DK / 4][kRows][4], l [kRows], reference [kRows].
template <int DK>
__device__ __forceinline__ float *part_at(const Plan &plan, int G, int slot, int g, int x) {
    return plan.parts + ((static_cast<int64_t>(slot) * G + g) * 2 + x) * (kRows * (DK + 2));
}

// Infinities and NaN that were taken out of partly visible tiles, of the keys
// this row sees, added to what the row has stored (once one is added, the sum is
// no number that rounding could change).
template <bool BF, typename T>
__device__ __noinline__ void add_odd(const AttendParams &p, const Work &w, int x, int pos, T *row) {
    const int lo = p.window > 0 ? max(pos + 1 - p.window, 0) : 0;
    for (int j = w.from[x]; j < w.to[x]; ++j) {
        if (!partly_seen(w, p.window, j)) continue;
        for (int key = max(j * kKeys, lo); key < min((j + 1) * kKeys, pos + 1); ++key) {
            const int64_t page = page_of(p.c, w.b, key);
            if (page < 0) continue;
            const unsigned short *v = static_cast<const unsigned short *>(p.c.v_cache) + page * p.c.vs[0] +
                                      (key % p.c.page) * p.c.vs[1] + w.g * p.c.vs[2];
            for (int d = 0; d < p.c.D; ++d) {
                const float f = bits_to_float(__ldg(v + d), BF ? kBF16 : kF16);
                if (fabsf(f) <= 3.402823466e38f) continue;
                if constexpr (sizeof(T) == 4) row[(d / 4) * (4 * kRows) + d % 4] += f;  // (a part's O)
                else row[d] = static_cast<T>(pack2<BF>(bits_to_float(row[d], BF ? kBF16 : kF16) + f, 0.f) & 0xffffu);
            }
        }
    }
}

__device__ __forceinline__ void store32(void *p, const uint32_t *u) {  // 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]),
                 "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// A row's scores of a key tile times `scale`, in place, each product rounded.  (A function of its
// own, which nearly no call comes to: in the softmax's loop, never run, it made 566 us of the 552
// that 32768 tokens in 16 prompts took without it; here 559.)
__device__ __noinline__ void scale_scores(uint32_t at, float scale) {
#pragma unroll 1
    for (int c = 0; c < kKeys; c += 16) {
        uint32_t r[16];
        tmem_ld16(at + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__fmul_rn(__uint_as_float(r[i]), scale));
        tmem_st16(at + c, r);
    }
    tmem_wait_st();
}

// DK: the head size, rounded up to 64; BF: bf16.
template <int DK, bool BF>
__global__ void __launch_bounds__(kThreads, 1) attend_tiles_kernel(const AttendParams p, const __grid_constant__ Maps maps, const Plan plan,
                                                                   int box, int flags, long long limit) {
    using LY = Layout<DK>;
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *const bars = reinterpret_cast<uint64_t *>(smem + LY::kBars);
    uint64_t *const full = bars + kRing, *const empty = full + LY::kBufs, *const clean = empty + LY::kBufs;
    Work *const ring = reinterpret_cast<Work *>(smem + LY::kWork);
    uint32_t *const tmem_at = reinterpret_cast<uint32_t *>(smem + LY::kMisc);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(smem + LY::kMisc) + 1;
    float2 *const stat = reinterpret_cast<float2 *>(smem + LY::kStat);
    // by piece of work and warp: were there values that are no numbers?
    volatile unsigned char *const odd = smem + LY::kMisc + 12;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const auto wait_on = [&](uint64_t *bar, uint32_t parity) { return sleep_on(bar, parity, limit); };
    if (warp == 8) tmem_alloc512(tmem_at);
    if (tid == 0) {
        *abort_flag = 0;
        for (int i = 0; i < kRing; ++i)
            mbar_init(&bars[i], i >= kUnitFree0 && i < kUnitEnd ? kReaders
                                : i >= kPFull0 && i < kOFull0 ? 4 : i >= kORead0 && i < kFinal ? 4 : 1);
        for (int i = 0; i < LY::kBufs; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 3), mbar_init(&clean[i], 2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    start_dependents();
    wait_for_prior();  // the plan
    bool ok = true;
    int nu = 0;  // pieces of work read
    const auto read_work = [&](const Work *&w) {
        if (!__all_sync(0xffffffffu, wait_on(&bars[kUnitFull0 + nu % kAhead], nu / kAhead & 1))) return false;
        w = &ring[nu % kWorks];
        if (lane == 0) mbar_arrive(&bars[kUnitFree0 + nu % kAhead]);
        ++nu;
        return true;
    };

    if (warp >= 8 && warp < 12) {
        registers_down<104>();
        if (warp == 9) {
            // ---------------- units and copies ----------------
            const int pieces = plan.head->pieces, units = pieces * p.c.G, tt = tile_tokens(p.c);
            const Piece *const list = plan.head->cuts > 0 ? plan.pieces : plan.units;
            int u = blockIdx.x, made = 0;
            // What the copies need of a piece; its place among the pieces kept.
            struct Load {
                int b, g, first, last, lo, end, at;
            };
            // The next piece, announced: false where a wait gave up.
            const auto next_work = [&](Load &l) {
                l.at = made % kWorks;
                Work w{};
                w.last = -1;  // (no key tiles: first > last)
                l.lo = INT_MAX, l.end = 0;
                if (u < units) {
                    const int i = u / p.c.G;
                    w.g = u - i * p.c.G;
                    const Piece q = list[i];
                    w.b = q.b;
                    w.first = q.last, w.last = q.first;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int t0 = (2 * q.pair + x) * tt;
                        w.toks[x] = max(min(tt, q.n - t0), 0);
                        w.row[x] = q.row0 + t0;
                        w.pos[x] = q.kv - q.n + t0;
                        key_tiles(p, w.pos[x], w.toks[x], w.from[x], w.to[x]);
                        w.from[x] = max(w.from[x], q.first);
                        w.to[x] = max(min(w.to[x], q.last), w.from[x]);
                        if (w.to[x] > w.from[x]) {
                            w.first = min(w.first, w.from[x]), w.last = max(w.last, w.to[x]);
                            l.end = max(l.end, w.pos[x] + w.toks[x]);
                            l.lo = min(l.lo, p.window > 0 ? w.pos[x] + 1 - p.window : 0);
                        }
                    }
                    if (w.last < w.first) w.first = w.last = 0;
                    w.part = q.part, w.parts = q.parts, w.slot = q.slot;
                    int nextu = 0;
                    if (lane == 0) nextu = atomicAdd(&plan.head->next, 1);
                    u = __shfl_sync(0xffffffffu, nextu, 0);
                }
                l.b = w.b, l.g = w.g, l.first = w.first, l.last = w.last;
                if (made >= kAhead && !__all_sync(0xffffffffu, wait_on(&bars[kUnitFree0 + made % kAhead], (made / kAhead - 1) & 1)))
                    return false;
                if (lane == 0) {
                    ring[made % kWorks] = w;
                    mbar_arrive(&bars[kUnitFull0 + made % kAhead]);
                }
                __syncwarp();
                ++made;
                return true;
            };
            const PageCopier<kKeys, LY::kPanels> pages(p.c, box);
            int n = 0, nq0 = 0, nq1 = 0;  // tiles copied; queries of A and B
            int buf = 0, turn = 0;
            const auto copy = [&](const CUtensorMap *map, int g, const auto &tile) {
                if (n >= LY::kBufs) ok = wait_on(&empty[buf], (turn & 1) ^ 1);
                ok = __all_sync(0xffffffffu, ok && !*abort_flag);
                if (!ok) return false;
                if (lane == 0) mbar_arrive_expect(&full[buf], tile.bytes);
                __syncwarp();
                pages.copy(tile, map, g, smem_addr(smem + LY::kBuf + buf * LY::kTile), &full[buf]);
                ++n;
                if (++buf == LY::kBufs) buf = 0, ++turn;
                return true;
            };
            const auto queries = [&](const Work &w, int x, int &nq) {
                if (w.to[x] <= w.from[x]) return true;
                if (nq > 0) ok = __all_sync(0xffffffffu, wait_on(&bars[kQFree0 + x], (nq - 1) & 1));
                if (!ok) return false;
                if (lane == 0) {
                    mbar_arrive_expect(&bars[kQFull0 + x], LY::kPanels * p.c.share * tt * 128);
                    for (int i = 0; i < LY::kPanels; ++i)
                        tma_load_3d(smem + x * LY::kTile + i * kPanel, &maps.q, 64 * i, w.g * p.c.share, static_cast<int>(w.row[x]),
                                    &bars[kQFull0 + x]);
                }
                __syncwarp();
                ++nq;
                return true;
            };
            // A piece is announced before the one ahead of it is copied, and a
            // tile's pages are looked up while the one before it is.
            Load w, after;
            ok = next_work(w);
            int page = ok && w.last > w.first ? pages.look_up(w.b, w.first, w.lo, w.end) : 0;
            while (ok && w.last >= 0) {
                if (!(ok = next_work(after))) break;
                for (int j = w.first; j < w.last; ++j) {
                    const auto tile = pages.find(page, j, w.lo, w.end);
                    const bool last = j + 1 == w.last;
                    if (!last || after.last > after.first)
                        page = pages.look_up(last ? after.b : w.b, last ? after.first : j + 1, last ? after.lo : w.lo, last ? after.end : w.end);
                    if (!copy(maps.cache.k, w.g, tile)) break;
                    if (j == w.first && (!queries(ring[w.at], 0, nq0) || !queries(ring[w.at], 1, nq1))) break;
                    if (!copy(maps.cache.v, w.g, tile)) break;
                }
                if (w.last <= w.first && after.last > after.first) page = pages.look_up(after.b, after.first, after.lo, after.end);
                w = after;
            }
            if (!ok && lane == 0) {
                flag(p.c.status, kDevTimeout);
                *abort_flag = 1;
            }
            // what was asked for has landed before the CTA retires
            if (lane == 0) {
                for (int i = 0; i < LY::kBufs && i < n; ++i) {
                    buf = buf == 0 ? LY::kBufs - 1 : buf - 1;
                    if (buf == LY::kBufs - 1) --turn;
                    wait_on(&full[buf], turn & 1);
                }
                if (nq0 > 0) wait_on(&bars[kQFull0], (nq0 - 1) & 1);
                if (nq1 > 0) wait_on(&bars[kQFull1], (nq1 - 1) & 1);
            }
            __syncwarp();
        } else if (warp == 8) {
            // ---------------- products ----------------
            // The warp runs this together, an elected lane issuing.  What matters
            // is little code between the waits: this warp is on the path of
            // every key tile, and shares its scheduler and instruction cache with
            // two that run long straight stretches.  With votes and checks around
            // each product a key tile took 4100 cycles, with the products
            // predicated in place of an elected branch (their descriptors formed
            // for each) 3300.  Loop counts and addresses are the same in every
            // lane and known to be (shuffled from lane 0), so that descriptors stay
            // in uniform registers.
            constexpr int bf = BF ? 1 : 0;
            const int ksteps = (p.c.D + 15) / 16, dims = (p.c.D + 15) / 16 * 16;
            const uint32_t id_s = idesc_f16(kRows, kKeys, 0, 0, bf), id_o = idesc_f16(kRows, dims, 0, 1, bf);
            const uint32_t s0 = smem_addr(smem), tm = __shfl_sync(0xffffffffu, tmem, 0);
            const Desc dQ(desc_k_sw128(s0)), dK(desc_k_sw128(s0 + LY::kBuf)), dV(desc_mn_sw128(s0 + LY::kBuf, kPanel));
            constexpr auto along_k = [](int k) { return static_cast<uint32_t>(((k / 4) * kPanel + (k % 4) * 32) >> 4); };
            constexpr auto along_mn = [](int k) { return static_cast<uint32_t>((k * 2048) >> 4); };
            // A wait that gives up only notes it, by lane: products of what is not
            // there yet stay within shared and tensor memory.  The lanes agree on it
            // once a key tile, ahead of every branch that it decides, and the loop
            // ends with that tile.
            const auto wait = [&](uint64_t *bar, int phase) {
                if (!mbar_try_wait(bar, phase & 1)) ok = wait_on(bar, phase & 1) && ok;
            };
            int kbuf = 0, kturn = 0, vbuf = 1, vturn = 0;
            const auto advance = [&](int &buf, int &turn) {
                buf += 2;
                if (buf >= LY::kBufs) buf -= LY::kBufs, ++turn;
            };
            int nq0 = 0, nq1 = 0, np0 = 0, np1 = 0, no0 = 0, no1 = 0;
            const auto uniform = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
            // (a tile that is known when this is compiled needs no shuffle)
            const auto of_tile = [&](auto t, uint32_t base, uint32_t step) {
                if constexpr (std::is_same<decltype(t), int>::value) return uniform(base + t * step);
                else return base + decltype(t)::value * step;
            };
            const auto scores = [&](auto t, bool keys_done, bool queries_done) {  // S of tile t
                tc_fence_after();
                Desc b = dK, a = dQ;
                b.lo = uniform(b.lo + kbuf * (LY::kTile >> 4));
                a.lo = of_tile(t, a.lo, LY::kTile >> 4);
                const uint32_t d = of_tile(t, tm + kColS, kKeys);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < DK / 16; ++i)
                        if (i < ksteps) mma(d, a + along_k(i), b + along_k(i), id_s, i > 0);
                    mma_commit(&bars[kSFull0 + t]);
                    if (keys_done) mma_commit(&empty[kbuf]);
                    if (queries_done) mma_commit(&bars[kQFree0 + t]);
                }
            };
            const auto outputs = [&](auto t, uint32_t acc, bool values_done) {  // O of tile t += P V
                tc_fence_after();
                Desc b = dV;
                b.lo = uniform(b.lo + vbuf * (LY::kTile >> 4));
                const uint32_t d = of_tile(t, tm + kColO, kKeys), a = of_tile(t, tm + kColS, kKeys);
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < kKeys / 16; ++i) mma_ts(d, a + 8 * i, b + along_mn(i), id_o, i > 0 ? 1u : acc);
                    mma_commit(&bars[kOFull0 + t]);
                    if (values_done) mma_commit(&empty[vbuf]);
                }
            };
            const auto release = [&](int buf) {
                if (elect_one()) mma_commit(&empty[buf]);
            };
            // A piece's key tiles as the products need them.
            struct Span {
                int from0, to0, from1, to1, first, last;
            };
            const auto next_span = [&](Span &s) {
                const Work *at;
                if (!read_work(at)) return false;
                s.from0 = uniform(at->from[0]), s.to0 = uniform(at->to[0]);
                s.from1 = uniform(at->from[1]), s.to1 = uniform(at->to[1]);
                s.first = uniform(at->first), s.last = uniform(at->last);
                return true;
            };
            // The scores of the next key tile, of this piece or the next, are
            // issued between the products of this one's P.  (A piece without keys
            // is not looked past before this one's are: its readers may wait for them.)
            const Known<0> A;
            const Known<1> B;
            Span w{}, n{};  // (w, j): the key tile whose P is next, if `some`; (n, jn): the one after it, if `more`
            bool some = false;
            int j = 0;
            for (;;) {
                // both tiles in the middle of their keys: nothing to decide
                if (some && j > max(w.from0, w.from1)) {
                    const int end = min(w.to0, w.to1) - 2;
                    for (; j < end && (ok = __all_sync(0xffffffffu, ok)); ++j) {
                        wait(&clean[vbuf], vturn);
                        wait(&bars[kPFull0], np0++);
                        outputs(A, 1, false);
                        wait(&full[kbuf], kturn);
                        scores(A, false, false);
                        wait(&bars[kPFull1], np1++);
                        outputs(B, 1, true);
                        scores(B, true, false);
                        advance(vbuf, vturn);
                        advance(kbuf, kturn);
                    }
                }
                int jn = j + 1;
                n = w;
                if (!some || jn >= w.last) {
                    if (!(ok = __all_sync(0xffffffffu, next_span(n) && ok))) break;
                    jn = n.first;
                }
                const bool more = n.last > n.first;
                if (some) wait(&clean[vbuf], vturn);
                if (more) wait(&full[kbuf], kturn);
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    const int from = t ? w.from1 : w.from0, to = t ? w.to1 : w.to0;
                    if (some && j >= from && j < to) {
                        wait(&bars[kPFull0 + t], t ? np1++ : np0++);
                        if (j == from) {  // O's columns are the last piece's until it is stored
                            const int no = t ? no1++ : no0++;
                            if (no > 0) wait(&bars[kORead0 + t], no - 1);
                        }
                        outputs(t, j > from, false);
                    }
                    const int nfrom = t ? n.from1 : n.from0, nto = t ? n.to1 : n.to0;
                    if (more && jn >= nfrom && jn < nto) {
                        if (jn == nfrom) wait(&bars[kQFull0 + t], t ? nq1 : nq0);
                        const bool done = jn + 1 == nto;
                        scores(t, false, done);
                        if (t) nq1 += done;
                        else nq0 += done;
                    }
                }
                if (some) {
                    release(vbuf);
                    advance(vbuf, vturn);
                }
                if (more) {
                    release(kbuf);
                    advance(kbuf, kturn);
                }
                w = n, j = jn, some = more;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok || w.last < 0) break;
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok && lane == 0) {
                flag(p.c.status, kDevTimeout);
                *abort_flag = 1;
            }
            // every product issued has completed before tensor memory is freed
            if (elect_one()) mma_commit(&bars[kFinal]);
            __syncwarp();
            wait_on(&bars[kFinal], 0);
            __syncwarp();
        } else {
            // ---------------- values of partly visible tiles ----------------
            // What no row sees becomes zeros, and so do infinities and NaN,
            // which a zero of P would spread to rows that do not see them: they
            // are added at the end to those that do.
            const Work *at;
            const int half = warp - 10;
            // They wait for every copy, keys and all, and pass on and release
            // every buffer, whether or not there is something to do: a wait for
            // a phase that is not the barrier's next one would mean nothing.
            // (The products wait for the values by `clean` alone; having waited
            // for the last key tile's, they know these two past any earlier use of
            // a buffer.)
            int buf = 0, turn = 0;
            const auto arrived = [&] { return __all_sync(0xffffffffu, wait_on(&full[buf], turn & 1)) != 0; };
            const auto release = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&clean[buf]), mbar_arrive(&empty[buf]);
                if (++buf == LY::kBufs) buf = 0, ++turn;
            };
            while ((ok = read_work(at)) && at->last >= 0) {
                const Work &w = *at;
                volatile unsigned char *const found_odd = &odd[2 * ((nu - 1) % kWorks) + half];
                if (lane == 0) *found_odd = 0;
                __syncwarp();
                int lo = INT_MAX, end = 0;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (w.to[x] > w.from[x]) {
                        end = max(end, w.pos[x] + w.toks[x]);
                        lo = min(lo, p.window > 0 ? w.pos[x] + 1 - p.window : 0);
                    }
                for (int j = w.first; j < w.last; ++j) {
                    if (!(ok = arrived())) break;  // the keys
                    release();
                    if (!(ok = arrived())) break;
                    if (__builtin_expect(partly_seen(w, p.window, j), 0)) {
                        unsigned char *const values = smem + LY::kBuf + buf * LY::kTile;
                        constexpr int kPieces = DK / 8, kAt = 32 / kPieces, kTurn = 2 * kAt;  // rows a warp, the two look at at once
                        bool found = false;
                        const int piece = lane % kPieces, mine = kAt * half + lane / kPieces;
                        const auto at_row = [&](int row) {
                            return reinterpret_cast<uint4 *>(values + (piece / 8) * kPanel + row * 128 + (((piece % 8) ^ (row & 7)) * 16));
                        };
                        // rows [r0, r1) of the tile, in turns of the two warps
                        const auto look = [&](int r0, int r1) {
#pragma unroll 1
                            for (int r = r0 + mine; r < r1; r += 4 * kTurn) {
                                uint4 v[4];
                                bool some = false;
#pragma unroll
                                for (int i = 0; i < 4; ++i) v[i] = r + i * kTurn < r1 ? *at_row(r + i * kTurn) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                                for (int i = 0; i < 4; ++i) some = any_odd<BF>(v[i]) || some;
                                if (__builtin_expect(some, 0)) {
                                    found = true;
#pragma unroll 1
                                    for (int row = r; row < min(r1, r + 4 * kTurn); row += kTurn) *at_row(row) = without_odd<BF>(*at_row(row));
                                }
                            }
                        };
                        const auto clear = [&](int r0, int r1) {
#pragma unroll 1
                            for (int r = r0 + mine; r < r1; r += kTurn) *at_row(r) = make_uint4(0u, 0u, 0u, 0u);
                        };
                        // what some row sees and another does not lies behind the first row's own key, or before
                        // the last one's window
                        const bool a = j >= w.from[0] && j < w.to[0], b = j >= w.from[1] && j < w.to[1];
                        const int pos = a ? w.pos[0] : w.pos[1], last = b ? w.pos[1] + w.toks[1] : w.pos[0] + w.toks[0];
                        const int seen = p.window > 0 ? min(max(last - p.window - j * kKeys, 0), kKeys) : 0;
                        const int r0 = min(max(lo - j * kKeys, 0), kKeys), r1 = min(max(end - j * kKeys, 0), kKeys);  // that some row sees
                        clear(0, r0);
                        clear(r1, kKeys);
#pragma unroll 1
                        for (int r = 0; r < 2; ++r) look(r ? max(max(pos + 1 - j * kKeys, 0), seen) : r0, r ? r1 : seen);
                        if (found) *found_odd = 1;
                        fence_proxy_async_smem();
                    }
                    release();
                }
                if (!ok) break;
            }
            if (!ok && lane == 0) {
                flag(p.c.status, kDevTimeout);
                *abort_flag = 1;
            }
        }
    } else if (warp >= 12) {
        registers_down<120>();
        // ---------------- outputs ----------------
        // Beside the next piece's products, whose first P V waits until O has
        // been read.  (By the softmax's own threads, a row each, a piece's end
        // took 8600 cycles where a key tile takes 2900.)
        const int warp_row = (warp & 3) * 32, m = warp_row + lane, tok = m / p.c.share, head = m - tok * p.c.share;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(warp_row) << 16);
        int done0 = 0, done1 = 0, tiles0 = 0, tiles1 = 0;  // of tile A, B: pieces with keys, key tiles
        const auto store = [&](const Work *at, int x) {
            const int from = at->from[x], to = at->to[x], toks = at->toks[x], pos = at->pos[x] + tok;
            if (toks <= 0) return true;
            const bool mine = tok < toks;
            const uint32_t colO = lanes + kColO + x * kKeys;
            float l = 0.f, ref = -INFINITY;
            if (to > from) {
                const int done = x ? done1++ : done0++, tiles = x ? tiles1 += to - from : tiles0 += to - from;
                if (!__all_sync(0xffffffffu, wait_on(&bars[kStat0 + x], done & 1))) return false;
                const float2 f = stat[x * kRows + m];
                l = f.x, ref = f.y;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kStatFree0 + x]);
                if (!__all_sync(0xffffffffu, wait_on(&bars[kOFull0 + x], (tiles - 1) & 1))) return false;
                tc_fence_after();
            }
            const auto o_read = [&] {
                if (to <= from) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kORead0 + x]);
            };
            const int slot = (nu - 1) % kWorks;
            const bool fix = (odd[2 * slot] | odd[2 * slot + 1]) != 0;
            const int64_t row = at->row[x] + tok;
            const int h = at->g * p.c.share + head;
            unsigned short *const out = static_cast<unsigned short *>(p.c.out) + row * p.c.os[0] + h * p.c.os[1];
            if (at->parts == 1) {
                const float inv = 1.f / l;
                const bool zero = to <= from || pos < 0, wide = flags & kWideOut;
                const uint64_t inv2 = pair(inv, inv);
#pragma unroll 1
                for (int c = 0; c < p.c.D; c += 32) {
                    uint32_t r[32], u[16];
                    if (to > from) {
                        tmem_ld32(colO + c, r);
                        tmem_wait_ld();
                    }
                    if (c + 32 >= p.c.D) o_read();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 f = unpair(mul2(pair(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), inv2));
                        u[i] = zero ? 0u : pack2<BF>(f.x, f.y);
                    }
                    // a row a thread: 32 bytes at a time where the rows lie for that, so that every sector is written at once
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        const int at = c + 2 * i;
                        if (!mine || at >= p.c.D) continue;
                        if (wide && at + 16 <= p.c.D) {
                            store32(out + at, u + i);
                        } else {
                            *reinterpret_cast<uint4 *>(out + at) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
                            if (at + 8 < p.c.D) *reinterpret_cast<uint4 *>(out + at + 8) = make_uint4(u[i + 4], u[i + 5], u[i + 6], u[i + 7]);
                        }
                    }
                }
                if (mine && p.lse) p.lse[row * p.c.H + h] = pos < 0 ? -INFINITY : lse_of(ref, l);
                if (__builtin_expect(fix, 0)) {
                    __syncwarp();
                    if (mine) add_odd<BF>(p, *at, x, pos, out);
                }
                return true;
            }
            // this part's O, l and reference, for the kernel that joins the parts
            float *const part = part_at<DK>(plan, p.c.G, at->slot + at->part, at->g, x);  // O as [DK / 4][kRows][4]
#pragma unroll 1
            for (int c = 0; c < DK; c += 16) {
                uint32_t r[16];
                if (to > from) {
                    tmem_ld16(colO + c, r);
                    tmem_wait_ld();
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0u;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(part + ((c / 4 + i) * kRows + m) * 4) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            }
            o_read();
            part[kRows * DK + m] = l;
            part[kRows * DK + kRows + m] = ref;
            if (__builtin_expect(fix, 0) && mine) add_odd<BF>(p, *at, x, pos, part + m * 4);
            return true;
        };
        const Work *at;
        while (ok && (ok = read_work(at)) && at->last >= 0)
#pragma unroll 1
            for (int x = 0; x < 2 && ok; ++x) ok = store(at, x);
        if (!ok && lane == 0) {
            flag(p.c.status, kDevTimeout);
            *abort_flag = 1;
        }
    } else {
        registers_up<144>();
        // ---------------- softmax (thread = row of tile x) ----------------
        const int x = warp >> 2, m = tid & (kRows - 1), tok = m / p.c.share;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t colS = lanes + kColS + x * kKeys, colO = lanes + kColO + x * kKeys;
        const float scale = p.scale * 1.4426950408889634f;
        int ns = 0, done = 0;  // score tiles seen (so many have been added to O); pieces with any
        const Work *at;
        while ((ok = read_work(at)) && at->last >= 0) {
            const int from = at->from[x], to = at->to[x], toks = at->toks[x], pos0 = at->pos[x], pos = pos0 + tok;
            const bool live = __any_sync(0xffffffffu, tok < toks);
            const int hi = pos + 1, lo = p.window > 0 ? pos + 1 - p.window : 0;  // it sees keys [lo, hi)
            float ref = -INFINITY, l = 0.f;
            float factor = scale;  // exponents are factor s - ref; 1 once a row of the warp has a coarse reference
            for (int j = from; j < to; ++j, ++ns) {
                if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[kSFull0 + x], ns & 1)))) break;
                tc_fence_after();
                if (live) {
                    if (__builtin_expect(!sees_all(p.window, pos0, toks, j), 0)) {
                        // (in place and in a loop: rarely run code must not stretch this path)
#pragma unroll 1
                        for (int c = 0; c < kKeys; c += 32) {
                            uint32_t r[32];
                            tmem_ld32(colS + c, r);
                            tmem_wait_ld();
                            const int h = hi - j * kKeys - c, o = lo - j * kKeys - c;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i >= h || i < o) r[i] = 0xff800000u;
                            tmem_st16(colS + c, r);
                            tmem_st16(colS + c + 16, r + 16);
                        }
                        tmem_wait_st();
                    }
                    // The scores are read twice, for their maximum and for P: held
                    // between the two they take the registers that the other groups need.
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    uint32_t s[2][32];
                    tmem_ld32(colS, s[0]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_wait_ld();
                        tmem_ld32(colS + (c < 3 ? 32 * c + 32 : 0), s[(c + 1) & 1]);  // (last: the first again, for P)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            top[(i >> 1) & 3] = max3(top[(i >> 1) & 3], __uint_as_float(s[c & 1][i]), __uint_as_float(s[c & 1][i + 1]));
                    }
                    const float now = __fmul_rn(fmaxf(max3(top[0], top[1], top[2]), top[3]), scale);
                    const bool moves = now - ref > kMost<BF>;  // (a difference: the sum would be rounded to the reference's step)
                    if (__builtin_expect(__any_sync(0xffffffffu, moves), 0)) {
                        const float level = fabsf(now) > kCoarse ? now : now - kLift<BF>, back = moves ? ex2(ref - level) : 1.f;
                        if (moves) ref = level, l *= back;
                        if (__any_sync(0xffffffffu, moves && fabsf(now) > kCoarse)) factor = 1.f;
                        if (j > from) {
                            if (!(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[kOFull0 + x], (ns - 1) & 1)))) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < DK; c += 16) {
                                uint32_t r[16];
                                tmem_ld16(colO + c, r);
                                tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * back);
                                tmem_st16(colO + c, r);
                            }
                        }
                    }
                    const float base = ref == -INFINITY ? 0.f : ref;
                    if (__builtin_expect(factor != scale, 0)) {
                        // scaled ones, rounded as the reference was: none of a row's is above its maximum then
                        tmem_wait_ld();
                        scale_scores(colS, scale);
                        tmem_ld32(colS, s[0]);
                    }
                    const uint64_t scale2 = pair(factor, factor), base2 = pair(-base, -base);
                    uint64_t add[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_wait_ld();
                        if (c < 3) tmem_ld32(colS + 32 * c + 32, s[(c + 1) & 1]);
                        uint32_t pr[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 e = unpair(fma2(pair(__uint_as_float(s[c & 1][2 * i]), __uint_as_float(s[c & 1][2 * i + 1])), scale2, base2));
                            const float a = ex2(e.x), b = ex2(e.y);
                            add[i & 3] = add2(add[i & 3], pair(a, b));
                            pr[i] = pack2<BF>(a, b);
                        }
                        tmem_st16(colS + 16 * c, pr);
                    }
                    const float2 sum = unpair(add2(add2(add[0], add[1]), add2(add[2], add[3])));
                    l += sum.x + sum.y;
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kPFull0 + x]);
            }
            if (!ok) break;
            if (to > from) {
                if (done > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[kStatFree0 + x], (done - 1) & 1)))) break;
                stat[x * kRows + m] = make_float2(l, ref);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[kStat0 + x]);
                ++done;
            }
        }
        if (!ok && lane == 0) {
            flag(p.c.status, kDevTimeout);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc512(tmem);
}

// The parts of units that were cut, joined: a CTA eight rows of a tile, four
// lanes of each warp a row, and a warp a quarter of the parts, whose sums are added in
// the order of the keys.  (By the CTA that stored a unit's last
// part, with one warp's loads in flight on a scheduler, a join took up to 140 us.)
template <int DK, bool BF>
__global__ void __launch_bounds__(128) attend_tiles_join_kernel(const AttendParams p, const Plan plan) {
    constexpr int kGroups = kRows / 8, kSlices = 4;
    wait_for_prior();
    const int lane = threadIdx.x & 31, G = p.c.G, tt = tile_tokens(p.c);
    const int64_t items = static_cast<int64_t>(plan.head->cuts) * G * 2 * kGroups;
    __shared__ float4 sums[kSlices - 1][DK / 16][32];
    __shared__ float ls[kSlices - 1][32];
    const int slice = threadIdx.x >> 5;
    for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
        const int group = static_cast<int>(i % kGroups), x = static_cast<int>(i / kGroups % 2), g = static_cast<int>(i / (2 * kGroups) % G);
        const Piece q = plan.pieces[plan.cuts[i / (2 * kGroups * G)]];
        const int m = 8 * group + lane / 4, tok = m / p.c.share, t0 = (2 * q.pair + x) * tt + tok;
        const bool there = tok < tt && t0 < q.n;
        float top = -INFINITY, sum = 0.f;
        float4 v[DK / 16] = {};  // columns 16 c + 4 (lane % 4) ...
        if (there) {
#pragma unroll 4
            for (int k = 0; k < q.parts; ++k) top = fmaxf(top, part_at<DK>(plan, G, q.slot + k, g, x)[kRows * (DK + 1) + m]);
            for (int k = q.parts * slice / kSlices; k < q.parts * (slice + 1) / kSlices; ++k) {
                const float *const part = part_at<DK>(plan, G, q.slot + k, g, x);
                const float ref = part[kRows * (DK + 1) + m], f = ref == -INFINITY ? 0.f : ex2(ref - top);
                sum += part[kRows * DK + m] * f;
#pragma unroll
                for (int c = 0; c < DK / 16; ++c) {  // (columns past the head size hold anything)
                    const float4 o = *reinterpret_cast<const float4 *>(part + ((4 * c + (lane & 3)) * kRows + m) * 4);
                    v[c].x += o.x * f, v[c].y += o.y * f, v[c].z += o.z * f, v[c].w += o.w * f;
                }
            }
        }
        if (slice > 0) {
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) sums[slice - 1][c][lane] = v[c];
            ls[slice - 1][lane] = sum;
        }
        __syncthreads();
        if (slice == 0 && there) {
#pragma unroll
            for (int k = 0; k < kSlices - 1; ++k) {
                sum += ls[k][lane];
#pragma unroll
                for (int c = 0; c < DK / 16; ++c) {
                    const float4 o = sums[k][c][lane];
                    v[c].x += o.x, v[c].y += o.y, v[c].z += o.z, v[c].w += o.w;
                }
            }
            const int pos = q.kv - q.n + t0;
            const float inv = 1.f / sum;
            const int64_t row = q.row0 + t0;
            const int h = g * p.c.share + (m - tok * p.c.share);
            unsigned short *const out = static_cast<unsigned short *>(p.c.out) + row * p.c.os[0] + h * p.c.os[1];
#pragma unroll
            for (int c = 0; c < DK / 16; ++c) {
                const int at = 16 * c + 4 * (lane & 3);
                if (at < p.c.D)
                    *reinterpret_cast<uint2 *>(out + at) =
                        pos < 0 ? make_uint2(0u, 0u) : make_uint2(pack2<BF>(v[c].x * inv, v[c].y * inv), pack2<BF>(v[c].z * inv, v[c].w * inv));
            }
            if (p.lse && (lane & 3) == 0) p.lse[row * p.c.H + h] = pos < 0 ? -INFINITY : lse_of(top, sum);
        }
        __syncthreads();  // `sums` are read
    }
}

constexpr int64_t kSlots = 1024;  // parts of cut units, all heads together

struct Split {
    int64_t units, slots;  // most units; most parts of cut ones (a head)
    uint64_t at_units, at_pieces, at_cuts, at_parts, bytes;
};
Split split_of(const PagedParams &c, int64_t max_kv_len) {
    const auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    Split s{};
    const int64_t pair = 2 * (kRows / c.share);
    s.units = c.rows / pair + c.nseq;  // >= sum of ceil(n / pair)
    // cut_of makes no parts of less than four key tiles but one, and no more of a unit than its longest
    // sequence has room for (a hint that is too small leaves units whole)
    const int64_t room = room_of(c), longest = max_kv_len > 0 && max_kv_len < room ? max_kv_len : room;
    const int64_t each = ((longest + kKeys - 1) / kKeys + 3) / 4 + 1, few = (each < kMaxParts ? each : kMaxParts) * s.units;
    // (a few key tiles are not worth cutting: 3 us for the joining kernel, a part's own cost)
    s.slots = max_kv_len > 0 && max_kv_len <= 8 * kKeys ? 0 : kSlots / c.G < few ? kSlots / c.G : few;
    const uint64_t dk = c.D <= 64 ? 64 : 128;
    s.at_units = up(sizeof(PlanHead));
    s.at_pieces = s.at_units + up(s.units * sizeof(Piece));
    s.at_cuts = s.at_pieces + up((s.slots > 0 ? s.units + s.slots : 0) * sizeof(Piece));
    s.at_parts = s.at_cuts + up(s.slots * sizeof(int32_t));
    s.bytes = s.at_parts + up(static_cast<uint64_t>(s.slots) * c.G * 2 * kRows * (dk + 2) * sizeof(float));
    return s;
}

template <int DK, bool BF>
cudaError_t launch_t(const AttendParams &p, int64_t max_kv_len, void *workspace, cudaStream_t stream) {
    // Before the maps: their encoder is a driver call and refuses a host thread
    // that has no context yet, which this one gives it.
    cudaError_t e = cudaFuncSetAttribute(attend_tiles_kernel<DK, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DK>::kBytes);
    if (e != cudaSuccess) return e;
    Maps maps;
    if (!encode_queries(&maps.q, p.c, kRows / p.c.share) || !encode_cache(&maps.cache, p.c, kKeys)) return cudaErrorInvalidValue;
    const int sms = device_sms();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const bool wide = reinterpret_cast<uintptr_t>(p.c.out) % 32 == 0 && (p.c.rows == 1 || p.c.os[0] % 16 == 0) && (p.c.H == 1 || p.c.os[1] % 16 == 0);
    const Split s = split_of(p.c, max_kv_len);
    unsigned char *const at = static_cast<unsigned char *>(workspace);
    Plan plan{};
    plan.head = reinterpret_cast<PlanHead *>(at);
    plan.units = reinterpret_cast<Piece *>(at + s.at_units);
    plan.pieces = reinterpret_cast<Piece *>(at + s.at_pieces);
    plan.cuts = reinterpret_cast<int32_t *>(at + s.at_cuts);
    plan.parts = reinterpret_cast<float *>(at + s.at_parts);
    plan.max_units = static_cast<int32_t>(s.units);
    plan.max_slots = static_cast<int32_t>(s.slots);
    attend_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, plan, sms);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    e = launch_after(attend_tiles_kernel<DK, BF>, dim3(sms), kThreads, Layout<DK>::kBytes, stream, p, maps, plan, least_box(p.c, kKeys),
                     wide ? kWideOut : 0, waits_of(p.c));
    if (e != cudaSuccess || s.slots == 0) return e;
    return launch_after(attend_tiles_join_kernel<DK, BF>, dim3(8 * sms), 128, 0, stream, p, plan);
}

}  // namespace

uint64_t attend_tiles_workspace(const PagedParams &c, int64_t max_kv_len) { return split_of(c, max_kv_len).bytes; }

cudaError_t launch_attend_tiles(const AttendParams &p, int64_t max_kv_len, void *workspace, cudaStream_t stream) {
    const bool bf = p.c.io_dtype == kBF16;
    if (p.c.D <= 64) return bf ? launch_t<64, true>(p, max_kv_len, workspace, stream) : launch_t<64, false>(p, max_kv_len, workspace, stream);
    return bf ? launch_t<128, true>(p, max_kv_len, workspace, stream) : launch_t<128, false>(p, max_kv_len, workspace, stream);
}

}  // namespace ssu
