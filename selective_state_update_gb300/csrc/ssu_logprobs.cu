// ssu_logprobs.cu -- log probabilities of given tokens, the entropy and the
// most likely alternatives, in one pass over the logits.
//
// Per row x of `vocab` logits, with m = max x:
//     s = sum exp(x - m),   t = sum (x - m) exp(x - m)
//     logprob = (x[token] - m) - ln s,   entropy = ln s - t / s
// and the top_k largest logits in order of (value, lowest index), each with
// its log probability.  s, t and m are fp32; a thread carries its own running
// maximum and rescales its sums when that grows:
//     d = m - m' <= 0:  s' = s e^d,  t' = (t + d s) e^d.
// The sums are taken in powers of two against M, m log2(e) rounded to fp32:
// x log2(e) - M is one FMA, and as M is the reference everywhere its rounding
// drops out.  The product would overflow beyond 2.3e38: logits below -1e38
// count as nothing, as they do beside any other, and a row that comes out with
// nothing or with a NaN (masked altogether, or with infinities) is gone through
// again with the difference x - m taken first.
//
// HBM-bound: every logit is read once.  A row is split over the CTAs of a
// cluster when there are few rows, and the parts are joined through
// distributed shared memory, so a call is one launch without a workspace.
// 4096 x 131072 bf16 with 20 alternatives: 214 us, 5.0 TB/s, 0.74 of the copy rate;
// without alternatives 194 us: a row's sums and search at its end take 1.3 and
// 1.6 us of its SM, and three CTAs an SM cover them only in part.
//
// The largest logits take no second pass.  While streaming, a thread only
// notes its largest value, which the softmax needs anyway, and the vectors it
// came from.  The k-th largest of the threads' maxima is a lower bound of the
// k-th largest logit, and only threads whose maximum reaches it can hold any
// logit that does: those threads' vectors (about k / threads of the row) are
// read again, out of L2.  What reaches the bound is collected, a little more
// than k as a rule, and placed by counting what is larger, by unique keys of
// value and index.  If too many tie with the bound for the collection, the
// threads' largest keys take the place of their values, which leaves k threads;
// if those alone hold too many, sorted lists of 32 keys a warp are kept instead.
#include <cooperative_groups.h>

#include "ssu_device.cuh"
#include "ssu_hybrid.h"

namespace ssu {

namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x by the special-function unit (relative error below 2^-22).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Values as integers in their order, never 0.  -0 equals 0, a NaN orders as
// -inf.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(fmaxf(x, -INFINITY) + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// Unique keys: larger values first, then lower indices; never 0.
__device__ __forceinline__ uint64_t make_key(float x, int idx) {
    return (static_cast<uint64_t>(ordered(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float key_value(uint64_t key) { return value_of(static_cast<uint32_t>(key >> 32)); }
__device__ __forceinline__ int key_index(uint64_t key) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}

// One compare-exchange step of a bitonic network over the lanes, descending
// where `desc`.
template <typename K>
__device__ __forceinline__ K exchange(K v, int m, bool desc) {
    const K o = __shfl_xor_sync(0xffffffffu, v, m);
    const bool upper = (threadIdx.x & m) != 0;
    return (v > o) == (upper != desc) ? v : o;
}
// The warp's 32 keys sorted downwards over the lanes.
template <typename K>
__device__ __forceinline__ K warp_sort(K v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
        for (int m = k >> 1; m > 0; m >>= 1) v = exchange(v, m, (lane & k) == 0);
    }
    return v;
}
// The 32 largest of two downward-sorted lists, sorted downwards.
template <typename K>
__device__ __forceinline__ K warp_merge(K a, K b) {
    const K r = __shfl_sync(0xffffffffu, b, 31 - (threadIdx.x & 31));
    K v = a > r ? a : r;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v = exchange(v, m, true);
    return v;
}
// The 32 largest of the CTA's keys, one a thread, sorted downwards at the
// start of `lists`; begins and ends with a barrier.
template <typename K>
__device__ __forceinline__ void largest_of_threads(K key, K *lists) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    lists[threadIdx.x] = warp_sort(key);
    __syncthreads();
#pragma unroll 1
    for (int half = kLpWarps / 2; half > 0; half >>= 1) {
        if (warp < half) lists[32 * warp + lane] = warp_merge(lists[32 * warp + lane], lists[32 * (warp + half) + lane]);
        __syncthreads();
    }
}

// Sums of one thread, warp or CTA: the reference m, s = sum 2^d and t = sum d
// 2^d of the exponents d = (x log2(e) - m), or with `unit` log2(e) those of a
// reference in the logits' own unit.
struct Stats {
    float m, s, t;
};
__device__ __forceinline__ void rescale(Stats &a, float m, float unit) {
    // never below -1e4: the power is zero long before, and the product with s
    // stays finite
    const float d = fmaxf((a.m - m) * unit, -1e4f);
    const float c = ex2(d);
    a.t = (a.t + d * a.s) * c;
    a.s *= c;
    a.m = m;
}
__device__ __forceinline__ Stats join(Stats a, Stats b, float unit) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m, unit);
    rescale(b, m, unit);
    return {m, a.s + b.s, a.t + b.t};
}

// Running maxima start at kFloor and elements are raised to kLow, below it:
// what is masked has the exponential zero, its product with the exponent is
// zero and not NaN, and a row of nothing else sums to zero.
constexpr float kFloor = -0.9e38f, kLow = -1e38f;
__device__ __forceinline__ float raise(float v) {  // a NaN stays
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(kLow));
    return r;
}

// VEC elements as loaded; the largest of them; as floats.
template <typename T>
struct Logits;
template <>
struct Logits<float> {
    uint4 u;
    __device__ __forceinline__ void none() { u.x = u.y = u.z = u.w = 0xff800000u; }
    __device__ __forceinline__ float largest() const {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    __device__ __forceinline__ void floats(float *v) const {
        StateChunk<float>::unpack(u, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = raise(v[j]);
    }
};
template <>
struct Logits<__half> {
    uint4 u;
    __device__ __forceinline__ void none() { u.x = u.y = u.z = u.w = 0xfc00fc00u; }
    __device__ __forceinline__ float largest() const {
        const __half2 *h = reinterpret_cast<const __half2 *>(&u);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ void floats(float *v) const {
        const __half2 *h = reinterpret_cast<const __half2 *>(&u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(h[j]);
            v[2 * j] = raise(f.x);
            v[2 * j + 1] = raise(f.y);
        }
    }
};
template <>
struct Logits<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void none() { u.x = u.y = u.z = u.w = 0xff80ff80u; }
    __device__ __forceinline__ float largest() const {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ void floats(float *v) const {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 low = __float2bfloat162_rn(kLow);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 c = __hmax2_nan(h[j], low);
            const uint32_t w = *reinterpret_cast<const uint32_t *>(&c);
            v[2 * j] = __uint_as_float(w << 16);
            v[2 * j + 1] = __uint_as_float(w & 0xffff0000u);
        }
    }
};

// A part of a row: vectors i < nv of VEC elements from element e0 on, and the
// `extra` elements outside the row's whole, aligned vectors -- those before
// (`head` of them, from element 0) and those after (from element `tail`).
// Vector i belongs to thread i % kLpThreads, extra e to thread e.
template <typename T>
struct Part {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    const T *x;
    int nv, e0, extra, head, tail;
    __device__ __forceinline__ Part(const LogprobParams &p, const T *row, int rank, int parts) : x(row) {
        int before = static_cast<int>((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T));
        if (before > p.vocab) before = p.vocab;
        const int all = (p.vocab - before) / VEC;
        const int v0 = static_cast<int>(static_cast<int64_t>(all) * rank / parts);
        nv = static_cast<int>(static_cast<int64_t>(all) * (rank + 1) / parts) - v0;
        e0 = before + v0 * VEC;
        head = rank == 0 ? before : 0;
        tail = before + all * VEC;
        extra = head + (rank == parts - 1 ? p.vocab - tail : 0);
    }
    __device__ __forceinline__ int extra_at(int e) const { return e < head ? e : tail + e - head; }
    __device__ __forceinline__ Logits<T> load(int i) const {
        Logits<T> l;
        l.u = *reinterpret_cast<const uint4 *>(x + e0 + i * VEC);
        return l;
    }
    __device__ __forceinline__ int element(int i, int j) const { return e0 + i * VEC + j; }
};

constexpr int kUnroll = 4;  // vectors a thread has in flight
constexpr int kMaxHits = 512;  // candidates collected before the sorted lists take over

// The sums over the CTA, in every lane of its first warp.
__device__ __forceinline__ Stats block_join(Stats a, Stats *wstats, float unit) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const Stats o = {__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
                         __shfl_xor_sync(0xffffffffu, a.t, off)};
        a = join(a, o, unit);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) wstats[warp] = a;
    __syncthreads();
    a = wstats[lane % kLpWarps];
#pragma unroll
    for (int off = kLpWarps / 2; off > 0; off >>= 1) {
        const Stats o = {__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
                         __shfl_xor_sync(0xffffffffu, a.t, off)};
        a = join(a, o, unit);
    }
    return a;
}

// The sums of a whole row with the difference taken before the product: for
// rows with nothing but values near the type's lowest, or with infinities.
template <typename T>
__device__ __noinline__ Stats careful_row(const T *x, int vocab, Stats *wstats) {
    Stats a = {-3.402823466e38f, 0.f, 0.f};
    for (int i = threadIdx.x; i < vocab; i += kLpThreads) {
        const float v = to_float(x[i]);
        if (v > a.m) rescale(a, v, kLog2e);
        const float d = (v - a.m) * kLog2e, e = ex2(d);
        a.s += e;
        a.t = fmaf(fmaxf(d, -1e4f), e, a.t);
    }
    return block_join(a, wstats, kLog2e);
}

// Shared memory of the search for the largest.
struct TopSearch {
    uint64_t lists[kLpThreads];
    uint64_t found[kMaxHits];
    int hits;
    uint64_t top[32];
};

// Collects the keys of a part that reach `bound`, from the lanes in `owners` of
// each warp (and every thread's extra element); true if they fitted, and then
// the 32 largest are in ts->top.
template <typename T>
__device__ __forceinline__ bool collect_top(const Part<T> &pt, uint64_t bound, bool owner, uint64_t extra_key, TopSearch *ts) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float low = bound == 0 ? -INFINITY : key_value(bound);
    const auto collect = [&](uint64_t k) {
        const int h = atomicAdd(&ts->hits, 1);
        if (h < kMaxHits) ts->found[h] = k;
    };
    if (tid == 0) ts->hits = 0;
    if (tid < 32) ts->top[tid] = 0;  // (with fewer than 32 the other places stay empty)
    __syncthreads();
    if (extra_key != 0 && extra_key >= bound) collect(extra_key);
    for (uint32_t rest = __ballot_sync(0xffffffffu, owner); rest; rest &= rest - 1) {
        for (int i = 32 * warp + __ffs(rest) - 1 + lane * kLpThreads; i < pt.nv; i += 32 * kLpThreads) {
            float v[Part<T>::VEC];
            StateChunk<T>::unpack(pt.load(i).u, v);
#pragma unroll
            for (int j = 0; j < Part<T>::VEC; ++j)
                if (!(v[j] < low)) {
                    const uint64_t k = make_key(v[j], pt.element(i, j));
                    if (k >= bound) collect(k);
                }
        }
    }
    __syncthreads();
    const int n = ts->hits;
    if (n > kMaxHits) return false;
    for (int i = tid; i < n; i += kLpThreads) {
        const uint64_t k = ts->found[i];
        int larger = 0;
        for (int j = 0; j < n; ++j) larger += ts->found[j] > k;
        if (larger < 32) ts->top[larger] = k;
    }
    return true;
}

// The same by the threads' largest keys, for rows with many ties.
template <typename T>
__device__ __noinline__ void tied_top(const Part<T> &pt, int top_k, float best, int best_i, uint64_t extra_key, TopSearch *ts) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t key = extra_key;
    if (best_i >= 0) {
        // the first element that is this thread's largest (where nothing is
        // above -inf, the first of all)
        int at = pt.element(best_i, 0);
        for (int u = kUnroll - 1; u >= 0 && best > -INFINITY; --u)
            for (int j = Part<T>::VEC - 1; j >= 0; --j)
                if (best_i + u * kLpThreads < pt.nv && to_float(pt.x[pt.element(best_i + u * kLpThreads, j)]) == best)
                    at = pt.element(best_i + u * kLpThreads, j);
        const uint64_t kb = make_key(best, at);
        key = kb > key ? kb : key;
    }
    largest_of_threads(key, ts->lists);
    const uint64_t bound = ts->lists[top_k - 1];
    if (collect_top(pt, bound, key >= bound, extra_key, ts)) return;
    // each warp keeps its owners' 32 largest in a sorted list over the lanes
    uint64_t mine = warp_sort(extra_key >= bound ? extra_key : uint64_t(0));
    for (uint32_t rest = __ballot_sync(0xffffffffu, key >= bound); rest; rest &= rest - 1) {
        for (int base = 32 * warp + __ffs(rest) - 1; base < pt.nv; base += 32 * kLpThreads) {
            const int i = base + lane * kLpThreads;
            for (int j = 0; j < Part<T>::VEC; ++j) {
                uint64_t k = i < pt.nv ? make_key(to_float(pt.x[pt.element(i, j)]), pt.element(i, j)) : 0;
                if (k < bound) k = 0;
                if (__any_sync(0xffffffffu, k != 0)) mine = warp_merge(mine, warp_sort(k));
            }
        }
    }
    largest_of_threads(mine, ts->lists);
    if (tid < 32) ts->top[tid] = ts->lists[tid];
}

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 1536 / kLpThreads) logprobs_kernel(const LogprobParams p, int parts) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    __shared__ Stats wstats[kLpWarps];
    __shared__ TopSearch ts;
    __shared__ Stats part_stats;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / parts;
    const int rank = static_cast<int>(blockIdx.x - row * parts);
    const T *const x = static_cast<const T *>(p.logits) + row * p.row_stride;
    const Part<T> pt(p, x, rank, parts);

    float m = kFloor;  // the largest so far
    Stats a = {kFloor * kLog2e, 0.f, 0.f};
    float best = -INFINITY;
    int best_i = tid < pt.nv ? tid : -1;  // the group of vectors with this thread's largest logit
    for (int i = tid; i < pt.nv; i += kUnroll * kLpThreads) {
        Logits<T> l[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (i + u * kLpThreads < pt.nv) l[u] = pt.load(i + u * kLpThreads);
            else l[u].none();
        }
        float vm = l[0].largest();
#pragma unroll
        for (int u = 1; u < kUnroll; ++u) vm = fmaxf(vm, l[u].largest());
        if (vm > best) {
            best = vm;
            best_i = i;
        }
        if (vm > m) {
            m = vm;
            rescale(a, m * kLog2e, 1.f);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float v[VEC];
            l[u].floats(v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = fmaf(v[j], kLog2e, -a.m), e = ex2(d);
                a.s += e;
                a.t = fmaf(d, e, a.t);
            }
        }
    }
    uint64_t key = 0;  // this thread's largest
    if (tid < pt.extra) {
        const float v = to_float(x[pt.extra_at(tid)]);
        key = make_key(v, pt.extra_at(tid));
        if (v > m) rescale(a, v * kLog2e, 1.f);
        const float d = fmaf(raise(v), kLog2e, -a.m), e = ex2(d);
        a.s += e;
        a.t = fmaf(d, e, a.t);
    }

    if (p.top_k > 0) {
        // by value: the bound's own ties are all collected
        uint32_t mine = best_i >= 0 ? ordered(best) : 0u;
        const uint32_t from_extra = static_cast<uint32_t>(key >> 32);
        mine = mine > from_extra ? mine : from_extra;
        uint32_t *lists = reinterpret_cast<uint32_t *>(ts.lists);
        largest_of_threads(mine, lists);
        const uint32_t bound = lists[p.top_k - 1];
        if (!collect_top(pt, static_cast<uint64_t>(bound) << 32, mine >= bound, key, &ts))
            tied_top(pt, p.top_k, best, best_i, key, &ts);
    }
    a = block_join(a, wstats, 1.f);  // (its barrier also completes ts.top)
    if (warp == 0) {
        if (lane == 0) part_stats = a;
    }
    if (parts > 1) cg::this_cluster().sync();
    else __syncthreads();
    if (rank == 0) {
        Stats b = part_stats;
        for (int c = 1; c < parts; ++c) b = join(b, *cg::this_cluster().map_shared_rank(&part_stats, c), 1.f);
        const bool careful = !(b.s > 0.f);  // (the same in every thread)
        if (careful) b = careful_row(x, p.vocab, wstats);
        if (warp == 0) {
            uint64_t top = p.top_k > 0 ? ts.top[lane] : 0;
            if (p.top_k > 0)
                for (int c = 1; c < parts; ++c) top = warp_merge(top, cg::this_cluster().map_shared_rank(ts.top, c)[lane]);
            const bool none = b.s == 0.f;  // every logit is -inf
            const float ls = log2f(b.s);
            const auto logprob = [&](float v) {
                if (none) return -INFINITY;
                if (careful) return (v - b.m) - kLn2 * ls;
                // far below the fast sums' range the logit itself is all that counts
                if (v < kLow && v > -INFINITY) return v - kLn2 * b.m;
                return kLn2 * (fmaf(v, kLog2e, -b.m) - ls);
            };
            if (lane == 0) {
                const int64_t tok = load_index(p.tokens, row, p.tok_is_i64);
                float lp = 0.f;
                if (tok >= 0 && tok < p.vocab) {
                    lp = logprob(to_float(x[tok]));
                } else if (tok != -1) {
                    flag(p.status, kDevBadEntry);
                    lp = __int_as_float(0x7fc00000);
                }
                p.logprob[row] = lp;
                p.entropy[row] = none ? 0.f : kLn2 * (ls - b.t / b.s);
            }
            if (lane < p.top_k) {
                const int64_t at = row * p.top_k + lane;
                const int idx = key_index(top);
                if (p.tok_is_i64) static_cast<int64_t *>(p.top_ids)[at] = idx;
                else static_cast<int32_t *>(p.top_ids)[at] = idx;
                p.top_logprob[at] = logprob(key_value(top));
            }
        }
    }
    // the others' shared memory stays until rank 0 has read it
    if (parts > 1) cg::this_cluster().sync();
}

template <typename T>
cudaError_t launch_lp_t(const LogprobParams &p, cudaStream_t stream) {
    // Two CTAs an SM are enough to split for: 256 rows of 100352 in one part
    // each take 22.9 us, in two 28.8; 40 rows in four parts 19.4 us, in two 24.6.
    int parts = 1;
    while (parts < kMaxCluster && p.rows * parts * 2 <= 304) parts *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows * parts));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(parts);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p, parts);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams &p, cudaStream_t stream) {
    switch (p.dtype) {
    case kF32: return launch_lp_t<float>(p, stream);
    case kF16: return launch_lp_t<__half>(p, stream);
    case kBF16: return launch_lp_t<__nv_bfloat16>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ssu
