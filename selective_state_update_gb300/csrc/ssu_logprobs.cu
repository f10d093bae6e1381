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
// drops out -- as long as it is small: it is the largest logit's exponent, and
// from |M| = 2^31 on may overflow the power.  Logits below -1e38 count as nothing,
// as they do beside any other.  A row whose |M| is above 2^26 (logits of 4.6e7; a
// row that a mask covers altogether), or that comes out with nothing or with a
// NaN, is gone through again with the difference x - m taken first.
//
// HBM-bound: every logit is read once.  A row is split over the CTAs of a
// cluster when there are few rows, and the parts are joined through
// distributed shared memory, so a call is one launch without a workspace.
// 4096 x 131072 bf16 with 20 alternatives: 187 us, 5.7 TB/s, 0.85 of the copy rate;
// without alternatives 166 us.  A row's end (sums, search) leaves its CTA's loads
// idle, so CTAs are small and many: of 512 threads, three an SM, four vectors in
// flight a thread it took 208 us, of 256 threads, six an SM 192, four an SM with
// eight vectors 188.
//
// The largest logits take no second pass.  While streaming, a thread notes its
// largest value, which the softmax needs anyway, and that of each group of
// vectors that it had in flight at once.  Threads 64 apart form a set; the k-th
// largest of the 64 sets' maxima is a lower bound of the k-th largest logit, and
// hardly more than k groups reach it (the k-th largest of the threads' maxima is
// a closer bound, but sorting all of them costs more).  Those groups are read
// again, all at once; what reaches the bound is collected and placed by
// counting what is larger, by unique keys of value and index.  (Reading all of
// such a thread's vectors again, one thread after the other, took 6 us more of
// the 188.)  If too many tie with the bound for the collection, the threads'
// largest keys take the place of their values, which leaves k threads; if those
// alone hold too many, sorted lists of 32 keys a warp are kept instead.
#include <cooperative_groups.h>

#include "ssu_device.cuh"
#include "ssu_hybrid.h"

namespace ssu {

namespace {

namespace cg = cooperative_groups;

constexpr int kLpSmThreads = 1024;  // resident a SM
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
template <int NT, typename K>
__device__ __forceinline__ void largest_of_threads(K key, K *lists) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    lists[threadIdx.x] = warp_sort(key);
    __syncthreads();
#pragma unroll 1
    for (int half = NT / 64; half > 0; half >>= 1) {
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
// The largest reference whose rounding (at most 4 there) leaves the sums exact.
constexpr float kMostReference = 67108864.f;
// Sums against a larger one may have overflowed.  They are nothing beside a
// smaller one, and not looked at where the row's own is no smaller; a NaN among
// the logits stays.
__device__ __forceinline__ void drop_unusable(Stats &a) {
    if (fabsf(a.m) > kMostReference) a.s = a.t = a.s == a.s ? 0.f : a.s;
}
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
// Vector i belongs to thread i % NT, extra e to thread e.
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

constexpr int kUnroll = 8;  // vectors a thread has in flight: a group
constexpr int kMaxGroups = 8;  // largest values noted a thread
constexpr int kMaxHits = 256;  // candidates collected before the sorted lists take over

// The sums over the CTA, in every lane of its first warp.
template <int NT>
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
    a = wstats[lane % (NT / 32)];
#pragma unroll
    for (int off = NT / 64; off > 0; off >>= 1) {
        const Stats o = {__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
                         __shfl_xor_sync(0xffffffffu, a.t, off)};
        a = join(a, o, unit);
    }
    return a;
}

// The sums of a whole row with the difference taken before the product: for
// rows whose largest logit is large in size, or with infinities.
template <typename T, int NT>
__device__ __noinline__ Stats careful_row(const T *x, int vocab, Stats *wstats) {
    Stats a = {-3.402823466e38f, 0.f, 0.f};
    for (int i = threadIdx.x; i < vocab; i += NT) {
        const float v = to_float(x[i]);
        if (v > a.m) rescale(a, v, kLog2e);
        const float d = (v - a.m) * kLog2e, e = ex2(d);
        a.s += e;
        a.t = fmaf(fmaxf(d, -1e4f), e, a.t);
    }
    return block_join<NT>(a, wstats, kLog2e);
}

// Shared memory of the search for the largest.  `groups` holds the largest of
// every 1 << shift groups of kUnroll vectors, in order, for each thread.
template <int NT>
struct TopSearch {
    uint64_t lists[NT];
    uint64_t found[kMaxHits];
    uint32_t spots[kMaxHits];
    float groups[kMaxGroups][NT];
    int hits, nspots;
    uint32_t bound;
    uint64_t top[32];
};

// Collects the keys of a part that reach `bound`, from the groups of the
// threads that are `owner` (and every thread's extra element); true if they
// fitted, and then the 32 largest are in ts->top.  The counters are zero and
// ts->top is empty before.
template <typename T, int NT>
__device__ __forceinline__ bool collect_top(const Part<T> &pt, int shift, uint64_t bound, bool owner, uint64_t extra_key,
                                            TopSearch<NT> *ts) {
    const int tid = threadIdx.x;
    const float low = bound == 0 ? -INFINITY : key_value(bound);
    const auto collect = [&](uint64_t k) {
        const int h = atomicAdd(&ts->hits, 1);
        if (h < kMaxHits) ts->found[h] = k;
    };
    if (extra_key != 0 && extra_key >= bound) collect(extra_key);
    if (owner) {
        for (int g = 0; tid + (g << shift) * (kUnroll * NT) < pt.nv; ++g) {
            if (ts->groups[g][tid] < low) continue;
            const int h = atomicAdd(&ts->nspots, 1);
            if (h < kMaxHits) ts->spots[h] = static_cast<uint32_t>(g * NT + tid);
        }
    }
    __syncthreads();
    const int spots = ts->nspots;
    if (spots > kMaxHits) return false;
    for (int w = tid / kUnroll; w < spots; w += NT / kUnroll) {
        const int g = static_cast<int>(ts->spots[w]) / NT, owner_tid = static_cast<int>(ts->spots[w]) % NT;
        int i = owner_tid + ((g << shift) * kUnroll + tid % kUnroll) * NT;
        for (int r = 0; r < 1 << shift && i < pt.nv; ++r, i += kUnroll * NT) {
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
    for (int i = tid; i < n; i += NT) {
        const uint64_t k = ts->found[i];
        int larger = 0;
        for (int j = 0; j < n; ++j) larger += ts->found[j] > k;
        if (larger < 32) ts->top[larger] = k;
    }
    return true;
}

// The same by the threads' largest keys, for rows with many ties.
template <typename T, int NT>
__device__ __noinline__ void tied_top(const Part<T> &pt, int shift, int top_k, float best, int best_i, uint64_t extra_key,
                                     TopSearch<NT> *ts) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t key = extra_key;
    if (best_i >= 0) {
        // the first element that is this thread's largest (where nothing is
        // above -inf, the first of all)
        int at = pt.element(best_i, 0);
        for (int u = kUnroll - 1; u >= 0 && best > -INFINITY; --u)
            for (int j = Part<T>::VEC - 1; j >= 0; --j)
                if (best_i + u * NT < pt.nv && to_float(pt.x[pt.element(best_i + u * NT, j)]) == best)
                    at = pt.element(best_i + u * NT, j);
        const uint64_t kb = make_key(best, at);
        key = kb > key ? kb : key;
    }
    __syncthreads();
    if (tid == 0) ts->hits = ts->nspots = 0;
    largest_of_threads<NT>(key, ts->lists);
    const uint64_t bound = ts->lists[top_k - 1];
    if (collect_top(pt, shift, bound, key >= bound, extra_key, ts)) return;
    // each warp keeps its owners' 32 largest in a sorted list over the lanes
    uint64_t mine = warp_sort(extra_key >= bound ? extra_key : uint64_t(0));
    for (uint32_t rest = __ballot_sync(0xffffffffu, key >= bound); rest; rest &= rest - 1) {
        for (int base = 32 * warp + __ffs(rest) - 1; base < pt.nv; base += 32 * NT) {
            const int i = base + lane * NT;
            for (int j = 0; j < Part<T>::VEC; ++j) {
                uint64_t k = i < pt.nv ? make_key(to_float(pt.x[pt.element(i, j)]), pt.element(i, j)) : 0;
                if (k < bound) k = 0;
                if (__any_sync(0xffffffffu, k != 0)) mine = warp_merge(mine, warp_sort(k));
            }
        }
    }
    largest_of_threads<NT>(mine, ts->lists);
    if (tid < 32) ts->top[tid] = ts->lists[tid];
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, kLpSmThreads / NT) logprobs_kernel(const LogprobParams p, int parts) {
    constexpr int VEC = 16 / static_cast<int>(sizeof(T));
    __shared__ Stats wstats[(NT / 32)];
    __shared__ TopSearch<NT> ts;
    __shared__ Stats part_stats;
    __shared__ alignas(8) int32_t token[2];  // low half first
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / parts;
    const int rank = static_cast<int>(blockIdx.x - row * parts);
    const T *const x = static_cast<const T *>(p.logits) + row * p.row_stride;
    const Part<T> pt(p, x, rank, parts);

    // The token is asked for now, by a copy that holds up no warp, and its
    // logit before the search, so that the row's end waits for neither.
    if (rank == 0 && tid == 0) {
        const unsigned to = static_cast<unsigned>(__cvta_generic_to_shared(token));
        if (p.tok_is_i64)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(static_cast<const int64_t *>(p.tokens) + row) : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(static_cast<const int32_t *>(p.tokens) + row) : "memory");
    }
    int shift = 0;
    while ((pt.nv - 1) / (kUnroll * NT) >> shift >= kMaxGroups) ++shift;

    float m = kFloor;  // the largest so far
    Stats a = {kFloor * kLog2e, 0.f, 0.f};
    float best = -INFINITY;
    int best_i = tid < pt.nv ? tid : -1;  // the group of vectors with this thread's largest logit
    float group = -INFINITY;
    for (int i = tid, step = 0; i < pt.nv; i += kUnroll * NT, ++step) {
        Logits<T> l[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (i + u * NT < pt.nv) l[u] = pt.load(i + u * NT);
            else l[u].none();
        }
        float vm = l[0].largest();
#pragma unroll
        for (int u = 1; u < kUnroll; ++u) vm = fmaxf(vm, l[u].largest());
        group = (step & ((1 << shift) - 1)) == 0 ? vm : fmaxf(group, vm);
        ts.groups[step >> shift][tid] = group;
        if (vm > best) {
            best = vm;
            best_i = i;
        }
        if (vm > m) {
            m = vm;
            drop_unusable(a);
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
        if (v > m) {
            drop_unusable(a);
            rescale(a, v * kLog2e, 1.f);
        }
        const float d = fmaf(raise(v), kLog2e, -a.m), e = ex2(d);
        a.s += e;
        a.t = fmaf(d, e, a.t);
    }
    drop_unusable(a);

    int64_t tok = -1;
    float tok_x = 0.f;
    if (rank == 0 && tid == 0) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        tok = p.tok_is_i64 ? *reinterpret_cast<const volatile int64_t *>(token) : *static_cast<const volatile int32_t *>(token);
        if (tok >= 0 && tok < p.vocab) tok_x = to_float(x[tok]);
    }
    if (p.top_k > 0) {
        // Threads 64 apart are a set; the k-th largest of the sets' largest is a
        // bound.  By value: the bound's own ties are all collected.
        uint32_t mine = best_i >= 0 ? ordered(best) : 0u;
        const uint32_t from_extra = static_cast<uint32_t>(key >> 32);
        mine = mine > from_extra ? mine : from_extra;
        uint32_t *lists = reinterpret_cast<uint32_t *>(ts.lists);
        lists[tid] = mine;
        if (tid == 0) ts.hits = ts.nspots = 0;
        if (tid < 32) ts.top[tid] = 0;  // (with fewer than 32 the other places stay empty)
        __syncthreads();
        if (warp == 0) {
            uint32_t s0 = lists[lane], s1 = lists[lane + 32];
#pragma unroll
            for (int j = 64; j < NT; j += 64) {
                s0 = max(s0, lists[lane + j]);
                s1 = max(s1, lists[lane + 32 + j]);
            }
            const uint32_t sorted = warp_merge(warp_sort(s0), warp_sort(s1));
            if (lane == p.top_k - 1) ts.bound = sorted;
        }
        __syncthreads();
        const uint32_t bound = ts.bound;
        if (!collect_top(pt, shift, static_cast<uint64_t>(bound) << 32, mine >= bound, key, &ts))
            tied_top(pt, shift, p.top_k, best, best_i, key, &ts);
    }
    a = block_join<NT>(a, wstats, 1.f);  // (its barrier also completes ts.top)
    if (warp == 0) {
        if (lane == 0) part_stats = a;
    }
    if (parts > 1) cg::this_cluster().sync();
    else __syncthreads();
    if (rank == 0) {
        Stats b = part_stats;
        for (int c = 1; c < parts; ++c) b = join(b, *cg::this_cluster().map_shared_rank(&part_stats, c), 1.f);
        const bool careful = !(b.s > 0.f && fabsf(b.m) <= kMostReference);  // (the same in every thread)
        if (careful) b = careful_row<T, NT>(x, p.vocab, wstats);
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
                float lp = 0.f;
                if (tok >= 0 && tok < p.vocab) {
                    lp = logprob(tok_x);
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

template <typename T, int NT>
cudaError_t launch_lp_t(const LogprobParams &p, int parts, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.rows * parts));
    cfg.blockDim = dim3(NT);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(parts);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, NT>, p, parts);
}

// Of 128 threads a CTA, eight an SM, where rows are short and enough to fill the
// SMs: 20000 rows of 32000 bf16 take 253 us (of 256 threads 300), 1216 18.5
// (20.3), 2432 of 65536 63 (66), but 304 of 32000 8.8 (7.9), 4096 of 131072 193 (186).
constexpr int64_t kSmallRows = 8 * 152, kSmallRowBytes = 131072;

template <typename T>
cudaError_t launch_lp(const LogprobParams &p, cudaStream_t stream) {
    // Two CTAs an SM are enough to split for: 256 rows of 100352 in one part each take
    // 15.2 us, in two 16.9; 40 rows in four parts 8.9, in eight 9.5 (100 rows of
    // 131072, 11.7 in two and 11.0 in four, are the other way round).
    int parts = 1;
    while (parts < kMaxCluster && p.rows * parts * 2 <= 304) parts *= 2;
    const int64_t bytes = static_cast<int64_t>(p.vocab) * static_cast<int64_t>(sizeof(T));
    if (p.rows >= kSmallRows && bytes <= kSmallRowBytes) return launch_lp_t<T, 128>(p, parts, stream);
    return launch_lp_t<T, 256>(p, parts, stream);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams &p, cudaStream_t stream) {
    switch (p.dtype) {
    case kF32: return launch_lp<float>(p, stream);
    case kF16: return launch_lp<__half>(p, stream);
    case kBF16: return launch_lp<__nv_bfloat16>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ssu
