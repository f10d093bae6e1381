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
//
// HBM-bound: every logit is read once.  A row is split over the CTAs of a
// cluster when there are few rows, and the parts are joined through
// distributed shared memory, so a call is one launch without a workspace.
//
// The largest logits take no second pass.  Keys (value made monotone, then
// the index downwards) are unique.  While streaming, a thread only notes its
// largest value (which the softmax needs anyway) and the vector it came from.
// The k-th largest of the threads' maxima is a lower bound of the k-th
// largest key, and only the k threads whose maximum reaches it can hold any
// key that does: those threads' vectors are read again (k / threads of the
// row, out of L2), and what reaches the bound goes through a sorted list of 32
// keys a warp.
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

// Unique keys: larger values first, then lower indices; never 0.  -0 equals
// 0, a NaN orders as -inf.
__device__ __forceinline__ uint64_t make_key(float x, int idx) {
    const float c = fmaxf(x, -INFINITY) + 0.f;
    const uint32_t b = __float_as_uint(c);
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return (static_cast<uint64_t>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(idx));
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int key_index(uint64_t key) {
    return static_cast<int>(0xffffffffu - static_cast<uint32_t>(key));
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int m) { return __shfl_xor_sync(0xffffffffu, v, m); }

// One compare-exchange step of a bitonic network over the lanes, descending
// where `desc`.
__device__ __forceinline__ uint64_t exchange(uint64_t v, int m, bool desc) {
    const uint64_t o = shfl_xor64(v, m);
    const bool upper = (threadIdx.x & m) != 0;
    return (v > o) == (upper != desc) ? v : o;
}
// The warp's 32 keys sorted downwards over the lanes.
__device__ __forceinline__ uint64_t warp_sort(uint64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
        for (int m = k >> 1; m > 0; m >>= 1) v = exchange(v, m, (lane & k) == 0);
    }
    return v;
}
// The 32 largest of two downward-sorted lists, sorted downwards.
__device__ __forceinline__ uint64_t warp_merge(uint64_t a, uint64_t b) {
    const uint64_t r = __shfl_sync(0xffffffffu, b, 31 - (threadIdx.x & 31));
    uint64_t v = a > r ? a : r;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v = exchange(v, m, true);
    return v;
}
// The 32 largest keys of `lists` downward-sorted lists of 32 (list i at
// base + 32 i) by one warp, sorted downwards over its lanes.
__device__ __forceinline__ uint64_t merge_lists(const uint64_t *base, int lists) {
    const int lane = threadIdx.x & 31;
    uint64_t v = base[lane];
    for (int i = 1; i < lists; ++i) v = warp_merge(v, base[32 * i + lane]);
    return v;
}

// Sums of one thread, warp or CTA.
struct Stats {
    float m, s, t;  // t in units of ln 2: sum of log2(e) (x - m) e^(x - m)
};
__device__ __forceinline__ void rescale(Stats &a, float m) {
    // never below -1e4: the exponential is zero long before, and the product
    // with s stays finite
    const float d = fmaxf((a.m - m) * kLog2e, -1e4f);
    const float c = ex2(d);
    a.t = (a.t + d * a.s) * c;
    a.s *= c;
    a.m = m;
}
__device__ __forceinline__ Stats join(Stats a, Stats b) {
    const float m = fmaxf(a.m, b.m);
    rescale(a, m);
    rescale(b, m);
    return {m, a.s + b.s, a.t + b.t};
}

template <typename T, int VEC>
__device__ __forceinline__ void unpack_vec(const T *p, float *v) {
    if constexpr (VEC == 1) v[0] = to_float(*p);
    else StateChunk<T>::unpack(*reinterpret_cast<const uint4 *>(p), v);
}

// A part of a row: the vectors [v0, v1) of VEC elements, and for the last
// part the `tail` elements that fill no vector, as vectors of one element
// after v1.  Vector v belongs to thread (v - v0) % kLpThreads.
template <typename T, int VEC>
struct Part {
    const T *x;
    int v0, v1, tail;
    __device__ __forceinline__ int count() const { return v1 - v0 + tail; }
    // element index of vector v0 + i, and how many elements it has
    __device__ __forceinline__ int first(int i) const {
        const int v = v0 + i;
        return v < v1 ? v * VEC : v1 * VEC + (v - v1);
    }
    __device__ __forceinline__ int size(int i) const { return v0 + i < v1 ? VEC : 1; }
};

template <typename T, int VEC>
__global__ void __launch_bounds__(kLpThreads) logprobs_kernel(const LogprobParams p, int parts) {
    __shared__ Stats wstats[kLpWarps];
    __shared__ uint64_t lists[kLpWarps * 32];
    __shared__ Stats part_stats;
    __shared__ uint64_t part_top[32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / parts;
    const int rank = static_cast<int>(blockIdx.x - row * parts);
    const int nvec = p.vocab / VEC;
    Part<T, VEC> pt;
    pt.x = static_cast<const T *>(p.logits) + row * p.row_stride;
    pt.v0 = static_cast<int>(static_cast<int64_t>(nvec) * rank / parts);
    pt.v1 = static_cast<int>(static_cast<int64_t>(nvec) * (rank + 1) / parts);
    pt.tail = rank == parts - 1 ? p.vocab - nvec * VEC : 0;
    const int n = pt.count();

    Stats a = {-3.402823466e38f, 0.f, 0.f};  // the floor keeps x - m defined for rows of -inf
    float best = -INFINITY;
    int best_i = -1;
    for (int i = tid; i < n; i += kLpThreads) {
        float v[VEC];
        if (pt.size(i) == VEC) {
            unpack_vec<T, VEC>(pt.x + pt.first(i), v);
        } else {
            v[0] = to_float(pt.x[pt.first(i)]);
#pragma unroll
            for (int j = 1; j < VEC; ++j) v[j] = -INFINITY;
        }
        float vm = -INFINITY;
#pragma unroll
        for (int j = 0; j < VEC; ++j) vm = fmaxf(vm, v[j]);
        if (vm > best || best_i < 0) {
            best = vm;
            best_i = i;
        }
        if (vm > a.m) rescale(a, vm);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float d = (v[j] - a.m) * kLog2e;
            const float e = ex2(d);
            a.s += e;
            a.t = fmaf(fmaxf(d, -1e4f), e, a.t);  // -inf * 0 would be NaN
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const Stats o = {__shfl_xor_sync(0xffffffffu, a.m, off), __shfl_xor_sync(0xffffffffu, a.s, off),
                         __shfl_xor_sync(0xffffffffu, a.t, off)};
        a = join(a, o);
    }
    if (lane == 0) wstats[warp] = a;

    if (p.top_k > 0) {
        // this thread's largest key
        uint64_t key = 0;
        if (best_i >= 0) {
            const int e0 = pt.first(best_i), ne = pt.size(best_i);
            for (int j = 0; j < ne; ++j) {
                const uint64_t kj = make_key(to_float(pt.x[e0 + j]), e0 + j);
                key = kj > key ? kj : key;
            }
        }
        lists[tid] = warp_sort(key);
        __syncthreads();
        // every warp: the 32 largest of the threads' maxima, their k-th as the bound
        const uint64_t owners = merge_lists(lists, kLpWarps);
        const uint64_t bound = __shfl_sync(0xffffffffu, owners, p.top_k - 1);
        __syncthreads();
        uint64_t mine = 0;  // this warp's list, sorted downwards over the lanes
        for (int o = warp; o < p.top_k; o += kLpWarps) {
            const uint64_t ok = __shfl_sync(0xffffffffu, owners, o);
            if (ok == 0) break;  // fewer threads with elements than k
            // the owner's vectors: those congruent to its own
            const int e = key_index(ok);
            const int i0 = (e < pt.v1 * VEC ? e / VEC : pt.v1 + (e - pt.v1 * VEC)) - pt.v0;
            for (int base = i0 % kLpThreads; base < n; base += 32 * kLpThreads) {
                const int i = base + lane * kLpThreads;
                const int ne = i < n ? pt.size(i) : 0;
                for (int j = 0; j < VEC; ++j) {
                    uint64_t kj = 0;
                    if (j < ne) kj = make_key(to_float(pt.x[pt.first(i) + j]), pt.first(i) + j);
                    if (kj < bound) kj = 0;
                    if (__any_sync(0xffffffffu, kj != 0)) mine = warp_merge(mine, warp_sort(kj));
                }
            }
        }
        lists[tid] = mine;
    }
    __syncthreads();
    if (warp == 0) {
        Stats b = lane < kLpWarps ? wstats[lane] : Stats{-3.402823466e38f, 0.f, 0.f};
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const Stats o = {__shfl_xor_sync(0xffffffffu, b.m, off), __shfl_xor_sync(0xffffffffu, b.s, off),
                             __shfl_xor_sync(0xffffffffu, b.t, off)};
            b = join(b, o);
        }
        if (lane == 0) part_stats = b;
        if (p.top_k > 0) part_top[lane] = merge_lists(lists, kLpWarps);
    }
    if (parts > 1) cg::this_cluster().sync();
    if (rank == 0 && warp == 0) {
        __syncwarp();
        Stats b = part_stats;
        uint64_t top = p.top_k > 0 ? part_top[lane] : 0;
        for (int c = 1; c < parts; ++c) {
            b = join(b, *cg::this_cluster().map_shared_rank(&part_stats, c));
            if (p.top_k > 0) top = warp_merge(top, cg::this_cluster().map_shared_rank(part_top, c)[lane]);
        }
        const bool none = b.s == 0.f;  // every logit is -inf
        const float lse = logf(b.s);
        if (lane == 0) {
            const int64_t tok = load_index(p.tokens, row, p.tok_is_i64);
            float lp = 0.f;
            if (tok >= 0 && tok < p.vocab) lp = none ? -INFINITY : (to_float(pt.x[tok]) - b.m) - lse;
            else if (tok != -1) {
                flag(p.status, kDevBadEntry);
                lp = __int_as_float(0x7fc00000);
            }
            p.logprob[row] = lp;
            p.entropy[row] = none ? 0.f : lse - kLn2 * (b.t / b.s);
        }
        if (lane < p.top_k) {
            const int64_t at = row * p.top_k + lane;
            const int idx = key_index(top);
            if (p.tok_is_i64) static_cast<int64_t *>(p.top_ids)[at] = idx;
            else static_cast<int32_t *>(p.top_ids)[at] = idx;
            p.top_logprob[at] = none ? -INFINITY : (key_value(top) - b.m) - lse;
        }
    }
    // the others' shared memory stays until rank 0 has read it
    if (parts > 1) cg::this_cluster().sync();
}

template <typename T, int VEC>
cudaError_t launch_lp(const LogprobParams &p, int parts, cudaStream_t stream) {
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
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T, VEC>, p, parts);
}

template <typename T>
cudaError_t launch_lp_t(const LogprobParams &p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    int parts = 1;
    while (parts < kMaxCluster && p.rows * parts * 2 <= 304) parts *= 2;
    const bool vec = p.row_stride % V == 0 && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0;
    return vec ? launch_lp<T, V>(p, parts, stream) : launch_lp<T, 1>(p, parts, stream);
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
