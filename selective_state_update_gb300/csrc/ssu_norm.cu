// ssu_norm.cu -- RMS norm of rows, with the residual's addition before it and
// an output in 16 or 32 bits or in E4M3 codes with scales.
//
// Per row of n = hidden columns:
//     r = x + residual               (fp32; residual_out = r rounded to x's type)
//     y = r * (mean(r^2) + eps)^-1/2 * w
// and either y rounded to x's type, or per group (the row, or 128 columns)
//     amax = max |y|;  scale = amax / 448;  code = E4M3(y * (448 / amax))
// (1 and 1 for a group of zeros), the read copy's E4M3 form.  The norm is
// taken of the fp32 sum, not of the stored residual: one rounding less.  Sum,
// mean and maximum are fp32.
//
// HBM-bound: every operand is read once and every output written once.  A CTA
// holds a row in registers between the two reductions (the sum of squares, the
// maximum), EPT elements a thread.  The grid is as large as the GPU holds at
// once; a CTA walks rows and has the next row's loads in flight while it reduces
// and stores the current one (rows of up to 4096 columns; wider ones leave no
// registers for it).  16384 x 8192 bf16 with residual and block scales: 155 us,
// 6.1 TB/s, 0.90 of the copy rate.
#include <type_traits>

#include "ssu_device.cuh"
#include "ssu_hybrid.h"

namespace ssu {

namespace {

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC consecutive elements (VEC = 1, or 16 bytes of T) as loaded, and as floats.
template <typename T, int VEC>
struct Raw {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void zero() { v = from_float<T>(0.f); }
    __device__ __forceinline__ void unpack(float *f) const { f[0] = to_float(v); }
};
template <typename T>
struct Raw<T, 16 / sizeof(T)> {
    static constexpr int kN = 16 / static_cast<int>(sizeof(T));
    union {
        uint4 v;
        T e[kN];
    };
    __device__ __forceinline__ Raw() {}
    // elements c of a row of n, c = col + i, that exist
    __device__ __forceinline__ void load_some(const T *row, int col, int n) {
        v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < kN; ++i)
            if (col + i >= 0 && col + i < n) e[i] = row[col + i];
    }
    __device__ __forceinline__ void load(const T *p) { v = ld_stream(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void unpack(float *f) const { StateChunk<T>::unpack(v, f); }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_some(T *row, int col, int n, const float *v) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        if (col + i >= 0 && col + i < n) row[col + i] = from_float<T>(v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float *v) {
    if constexpr (VEC == 1) {
        *p = from_float<T>(v[0]);
    } else {
        *reinterpret_cast<uint4 *>(p) = StateChunk<T>::pack(v);
    }
}
// VEC weights (any alignment of a vector's first element that its type has).
template <int VEC>
__device__ __forceinline__ void load_weight(const NormParams &p, int col, float *w) {
    if (p.weight_dtype == kF32) {
        const float *q = static_cast<const float *>(p.weight) + col;
        if constexpr (VEC == 1) {
            w[0] = __ldg(q);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(q + i));
                w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
            }
        }
        return;
    }
    const unsigned short *q = static_cast<const unsigned short *>(p.weight) + col;
    if constexpr (VEC == 1) {
        w[0] = bits_to_float(__ldg(q), p.weight_dtype);
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(q));  // only with 16-bit x: VEC == 8
        if (p.weight_dtype == kBF16) StateChunk<__nv_bfloat16>::unpack(u, w);
        else StateChunk<__half>::unpack(u, w);
    }
}

// Sum or maximum over the CTA; `part` holds one float per warp.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float *part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    v = lane < warps ? part[lane] : 0.f;  // maxima here are of magnitudes
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = MAX ? fmaxf(v, o) : v + o;
    }
    return v;
}

// Elements a thread holds by the row's width, and the threads that makes at
// most.  More of them make smaller CTAs, whose reductions are shorter and of
// which more rows are under way at once.  Measured on 2^27 bf16 elements with
// residual and block scales: width 2048 with 8 elements a thread 176 us, with 16
// 154; 4096 with 8 183, with 16 157; 8192 with 16 161, with 32 155 (16-bit output:
// 166 and 175); 16384 with 16 170, with 32 159; 1024 with 8 164.
constexpr int elements_per_thread(int hidden) { return hidden <= 1024 ? 8 : hidden <= 4096 ? 16 : 32; }
constexpr int ept_threads(int ept) { return ept == 8 ? 1024 / 8 : ept == 16 ? 4096 / 16 : kNormMaxHidden / 32; }

// T: element type of x; VEC: elements a load; EPT: elements a thread; RES:
// with a residual; LOOSE: rows that begin anywhere.  With VEC > 1 a loose row is
// still taken in aligned vectors (x, residual and outputs begin at the same
// place within one, `shift` elements in), the first and the last in part.
template <typename T, int VEC, int EPT, bool RES, bool LOOSE>
__global__ void __launch_bounds__(ept_threads(EPT), 1024 / ept_threads(EPT)) norm_kernel(const NormParams p) {
    constexpr int NV = EPT / VEC;
    constexpr bool kAhead = EPT < 32;  // a second row does not fit the registers of 1024 threads
    __shared__ float part[2][32];
    __shared__ int bmax[kNormMaxHidden / kNormBlock];  // LOOSE: the blocks' maxima (bits of non-negative floats)
    const int tid = threadIdx.x, nthr = blockDim.x;
    const auto shift_of = [&](int64_t row) {
        if constexpr (!LOOSE || VEC == 1) return 0;
        else return static_cast<int>(reinterpret_cast<uintptr_t>(static_cast<const T *>(p.x) + row * p.xs) / sizeof(T) % VEC);
    };
    const auto whole = [&](int col) { return !LOOSE || VEC == 1 ? col < p.hidden : col >= 0 && col + VEC <= p.hidden; };
    Raw<T, VEC> xr[NV], er[RES ? NV : 1];
    const auto fetch = [&](int64_t row) {
        const T *x = static_cast<const T *>(p.x) + row * p.xs;
        const T *res = RES ? static_cast<const T *>(p.residual) + row * p.rs : nullptr;
        const int shift = shift_of(row);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (tid + j * nthr) * VEC - shift;
            if (row < p.rows && whole(col)) {
                xr[j].load(x + col);
                if constexpr (RES) er[j].load(res + col);
            } else {
                xr[j].zero();
                if constexpr (RES) er[j].zero();
                if constexpr (LOOSE && VEC > 1) {
                    if (row < p.rows && col < p.hidden) {
                        xr[j].load_some(x, col, p.hidden);
                        if constexpr (RES) er[j].load_some(res, col, p.hidden);
                    }
                }
            }
        }
    };
    if (kAhead) fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        if (!kAhead) fetch(row);
        const int shift = shift_of(row);
        // a row of an output in T
        const auto store_row = [&](T *y, const float *v) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = (tid + j * nthr) * VEC - shift;
                if (whole(col)) store_vec<T, VEC>(y + col, v + j * VEC);
                else if (LOOSE && VEC > 1) store_some<T, VEC>(y, col, p.hidden, v + j * VEC);
            }
        };
        float r[EPT];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            xr[j].unpack(r + j * VEC);
            if constexpr (RES) {
                float e[VEC];
                er[j].unpack(e);
#pragma unroll
                for (int i = 0; i < VEC; ++i) r[j * VEC + i] += e[i];
            }
        }
        if (kAhead) fetch(row + gridDim.x);
        if constexpr (RES) store_row(static_cast<T *>(p.residual_out) + row * p.ros, r);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) ss = fmaf(r[i], r[i], ss);
        ss = block_reduce<false>(ss, part[0]);
        float inv = __frsqrt_rn(ss / static_cast<float>(p.hidden) + p.eps);
        if constexpr (sizeof(T) == 4 || std::is_same<T, __nv_bfloat16>::value) {
            if (ss > 3.402823466e38f) {
                // squares past fp32's range (values from 1e17 on): again of r 2^-80, beside which eps is nothing
                __syncthreads();  // `part` is read
                ss = 0.f;
#pragma unroll
                for (int i = 0; i < EPT; ++i) {
                    const float small = r[i] * 0x1p-80f;
                    ss = fmaf(small, small, ss);
                }
                ss = block_reduce<false>(ss, part[0]);
                inv = __frsqrt_rn(ss / static_cast<float>(p.hidden)) * 0x1p-80f;
            }
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (tid + j * nthr) * VEC - shift;
            float w[VEC];
            if constexpr (LOOSE) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    w[i] = 0.f;
                    if (col + i >= 0 && col + i < p.hidden) load_weight<1>(p, col + i, w + i);
                }
            } else if (col < p.hidden) {
                load_weight<VEC>(p, col, w);
            } else {
                continue;
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j * VEC + i] = r[j * VEC + i] * inv * w[i];
        }
        if (p.quant == kQuantNone) {
            store_row(static_cast<T *>(p.y) + row * p.ys, r);
            __syncthreads();  // `part` is read
            continue;
        }
        unsigned char *y = static_cast<unsigned char *>(p.y) + row * p.ys;
        // E4M3 codes of vector j, the factor of element i given
        const auto store_codes = [&](int j, auto factor) {
            const int col = (tid + j * nthr) * VEC - shift;
            const float *v = r + j * VEC;
            if (VEC > 1 && whole(col)) {
                uint32_t w[VEC / 4 + 1];
#pragma unroll
                for (int i = 0; i < VEC / 4; ++i)
                    w[i] = e4m3x2_codes(v[4 * i] * factor(4 * i), v[4 * i + 1] * factor(4 * i + 1)) |
                           (e4m3x2_codes(v[4 * i + 2] * factor(4 * i + 2), v[4 * i + 3] * factor(4 * i + 3)) << 16);
                if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(y + col) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint32_t *>(y + col) = w[0];
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (col + i >= 0 && col + i < p.hidden) y[col + i] = e4m3_code(v[i] * factor(i));
            }
        };
        if (p.quant == kQuantRow) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < EPT; ++i) m = fmaxf(m, fabsf(r[i]));
            m = block_reduce<true>(m, part[1]);
            if (tid == 0) p.scales[row] = shadow_scale_of(m);
            const float f = shadow_factor_of(m);
#pragma unroll
            for (int j = 0; j < NV; ++j) store_codes(j, [&](int) { return f; });
        } else {
            const int nblk = (p.hidden + kNormBlock - 1) / kNormBlock;
            float *scales = p.scales + row * nblk;
            if constexpr (LOOSE) {
                for (int b = tid; b < nblk; b += nthr) bmax[b] = 0;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int col = (tid + j * nthr) * VEC - shift;
                    // (a NaN counts as no magnitude, as in fmaxf)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (col + i >= 0 && col + i < p.hidden && r[j * VEC + i] == r[j * VEC + i])
                            atomicMax(&bmax[(col + i) / kNormBlock], __float_as_int(fabsf(r[j * VEC + i])));
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    const int col = (tid + j * nthr) * VEC - shift;
                    store_codes(j, [&](int i) {
                        const int c = min(max(col + i, 0), p.hidden - 1);
                        return shadow_factor_of(__int_as_float(bmax[c / kNormBlock]));
                    });
                }
                for (int b = tid; b < nblk; b += nthr) scales[b] = shadow_scale_of(__int_as_float(bmax[b]));
            } else {
                // 128 / VEC neighbouring lanes hold a block
                constexpr int L = kNormBlock / VEC;
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) m = fmaxf(m, fabsf(r[j * VEC + i]));
#pragma unroll
                    for (int off = L / 2; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                    const int col = (tid + j * nthr) * VEC;
                    if (col < p.hidden && tid % L == 0) scales[col / kNormBlock] = shadow_scale_of(m);
                    const float f = shadow_factor_of(m);
                    if (col < p.hidden) store_codes(j, [&](int) { return f; });
                }
            }
        }
        __syncthreads();  // `part` and `bmax` are read
    }
}

bool aligned(const void *q, int64_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; }

// CTAs of this kernel that the device holds at once, by device and threads (cached).
template <typename T, int VEC, int EPT, bool RES, bool LOOSE>
int resident(int threads) {
    static int cache[64][33];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    int *const kept = dev >= 0 && dev < 64 ? &cache[dev][threads / 32] : nullptr;
    int n = kept ? __atomic_load_n(kept, __ATOMIC_RELAXED) : 0;
    if (n == 0) {
        int sms = 0, per = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, norm_kernel<T, VEC, EPT, RES, LOOSE>, threads, 0) != cudaSuccess ||
            per <= 0)
            return 0;
        n = per * sms;
        if (kept) __atomic_store_n(kept, n, __ATOMIC_RELAXED);
    }
    return n;
}

template <typename T, int VEC, int EPT, bool RES, bool LOOSE>
cudaError_t launch_norm_r(const NormParams &p, cudaStream_t stream) {
    const int columns = p.hidden + (LOOSE ? VEC - 1 : 0);  // (whatever the shift)
    const int threads = ((columns + EPT - 1) / EPT + 31) / 32 * 32;
    const int most = resident<T, VEC, EPT, RES, LOOSE>(threads);
    if (most <= 0) return cudaErrorInvalidConfiguration;
    // as many rows for every CTA, or one less
    const int64_t turns = (p.rows + most - 1) / most;
    const unsigned grid = static_cast<unsigned>((p.rows + turns - 1) / turns);
    norm_kernel<T, VEC, EPT, RES, LOOSE><<<grid, threads, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename T, int VEC, int EPT, bool LOOSE>
cudaError_t launch_norm_k(const NormParams &p, cudaStream_t stream) {
    return p.residual ? launch_norm_r<T, VEC, EPT, true, LOOSE>(p, stream) : launch_norm_r<T, VEC, EPT, false, LOOSE>(p, stream);
}
template <typename T, int VEC, bool LOOSE>
cudaError_t launch_norm_v(const NormParams &p, cudaStream_t stream) {
    const int ept = elements_per_thread(p.hidden + (LOOSE ? VEC - 1 : 0));
    if (ept == 8) return launch_norm_k<T, VEC, 8, LOOSE>(p, stream);
    if (ept == 16) return launch_norm_k<T, VEC, 16, LOOSE>(p, stream);
    return launch_norm_k<T, VEC, 32, LOOSE>(p, stream);
}

// How the rows of the operands lie: all on 16-byte boundaries; all alike within
// 16 bytes, so that aligned vectors cover them; or neither, element by element
// (1001 rows of 2565 fp16 values: 9.3 us in vectors, 14.8 by element).
template <typename T>
cudaError_t launch_norm_t(const NormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    const int64_t ye = p.quant == kQuantNone ? sizeof(T) : 1;  // bytes of an output element
    const auto place = [](const void *q, int64_t size) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(q) / size % V); };
    const auto step = [&](int64_t stride) { return p.rows > 1 ? stride % V : 0; };
    const int64_t at = place(p.x, sizeof(T)), xstep = step(p.xs);
    const bool alike = reinterpret_cast<uintptr_t>(p.y) % ye == 0 && place(p.y, ye) == at && step(p.ys) == xstep &&
                       (!p.residual || (place(p.residual, sizeof(T)) == at && step(p.rs) == xstep &&
                                        place(p.residual_out, sizeof(T)) == at && step(p.ros) == xstep));
    const bool vec = alike && at == 0 && xstep == 0 && p.hidden % V == 0 && aligned(p.weight, 16) &&
                     (p.weight_dtype == kF32 || V == 8);
    if (vec) return launch_norm_v<T, V, false>(p, stream);
    if (alike && p.hidden + V - 1 <= kNormMaxHidden) return launch_norm_v<T, V, true>(p, stream);
    return launch_norm_v<T, 1, true>(p, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, cudaStream_t stream) {
    switch (p.dtype) {
    case kF32: return launch_norm_t<float>(p, stream);
    case kF16: return launch_norm_t<__half>(p, stream);
    case kBF16: return launch_norm_t<__nv_bfloat16>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ssu
