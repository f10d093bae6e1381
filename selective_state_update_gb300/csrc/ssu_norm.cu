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
// HBM-bound: every operand is read once and every output written once.  One
// CTA holds a row in registers between the two reductions (the sum of
// squares, the maximum), kEpt elements a thread.
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

// VEC consecutive elements <-> floats (VEC = 1, or 16 bytes of T).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float *v) {
    if constexpr (VEC == 1) {
        v[0] = to_float(*p);
    } else {
        StateChunk<T>::unpack(ld_stream(p), v);
    }
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

// T: element type of x; VEC: elements a load; EPT: elements a thread.
template <typename T, int VEC, int EPT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
    constexpr int NV = EPT / VEC;
    __shared__ float part[2][32];
    __shared__ int bmax[kNormMaxHidden / kNormBlock];  // VEC == 1: the blocks' maxima (bits of non-negative floats)
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, nthr = blockDim.x;
    const T *x = static_cast<const T *>(p.x) + row * p.xs;
    const T *res = p.residual ? static_cast<const T *>(p.residual) + row * p.rs : nullptr;
    float r[EPT];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (tid + j * nthr) * VEC;
        if (col < p.hidden) {
            load_vec<T, VEC>(x + col, r + j * VEC);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j * VEC + i] = 0.f;
        }
    }
    if (res) {
        float e[EPT];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (tid + j * nthr) * VEC;
            if (col < p.hidden) {
                load_vec<T, VEC>(res + col, e + j * VEC);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) e[j * VEC + i] = 0.f;
            }
        }
        T *ro = static_cast<T *>(p.residual_out) + row * p.ros;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (tid + j * nthr) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j * VEC + i] += e[j * VEC + i];
            if (col < p.hidden) store_vec<T, VEC>(ro + col, r + j * VEC);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) ss = fmaf(r[i], r[i], ss);
    ss = block_reduce<false>(ss, part[0]);
    const float inv = __frsqrt_rn(ss / static_cast<float>(p.hidden) + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (tid + j * nthr) * VEC;
        if (col < p.hidden) {
            float w[VEC];
            load_weight<VEC>(p, col, w);
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j * VEC + i] = r[j * VEC + i] * inv * w[i];
        }
    }
    if (p.quant == kQuantNone) {
        T *y = static_cast<T *>(p.y) + row * p.ys;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int col = (tid + j * nthr) * VEC;
            if (col < p.hidden) store_vec<T, VEC>(y + col, r + j * VEC);
        }
        return;
    }
    // Maxima of the groups, per vector j.
    float amax[NV];
    if (p.quant == kQuantRow) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) m = fmaxf(m, fabsf(r[i]));
        m = block_reduce<true>(m, part[1]);
#pragma unroll
        for (int j = 0; j < NV; ++j) amax[j] = m;
        if (tid == 0) p.scales[row] = shadow_scale_of(m);
    } else {
        const int nblk = (p.hidden + kNormBlock - 1) / kNormBlock;
        float *scales = p.scales + row * nblk;
        if constexpr (VEC == 1) {
            for (int b = tid; b < nblk; b += nthr) bmax[b] = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = tid + j * nthr;
                // a NaN counts as no magnitude, as in fmaxf
                if (col < p.hidden && r[j] == r[j]) atomicMax(&bmax[col / kNormBlock], __float_as_int(fabsf(r[j])));
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int col = tid + j * nthr;
                amax[j] = col < p.hidden ? __int_as_float(bmax[col / kNormBlock]) : 0.f;
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
                amax[j] = m;
                const int col = (tid + j * nthr) * VEC;
                if (col < p.hidden && tid % L == 0) scales[col / kNormBlock] = shadow_scale_of(m);
            }
        }
    }
    unsigned char *y = static_cast<unsigned char *>(p.y) + row * p.ys;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int col = (tid + j * nthr) * VEC;
        if (col >= p.hidden) continue;
        const float f = shadow_factor_of(amax[j]);
        if constexpr (VEC == 1) {
            y[col] = e4m3_code(r[j] * f);
        } else {
            uint32_t w[VEC / 4];
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float *v = r + j * VEC + 4 * i;
                w[i] = e4m3x2_codes(v[0] * f, v[1] * f) | (e4m3x2_codes(v[2] * f, v[3] * f) << 16);
            }
            if constexpr (VEC == 8) *reinterpret_cast<uint2 *>(y + col) = make_uint2(w[0], w[1]);
            else *reinterpret_cast<uint32_t *>(y + col) = w[0];
        }
    }
}

bool aligned(const void *q, int64_t a) { return reinterpret_cast<uintptr_t>(q) % a == 0; }

template <typename T>
cudaError_t launch_norm_t(const NormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    // 16-byte accesses need every row of every operand to start on its vector's boundary
    const int64_t ye = p.quant == kQuantNone ? sizeof(T) : 1;  // bytes of an output element
    const bool vec = p.hidden % V == 0 && p.xs % V == 0 && aligned(p.x, 16) && p.ys % V == 0 && aligned(p.y, V * ye) &&
                     aligned(p.weight, 16) && (p.weight_dtype == kF32 || V == 8) &&
                     (!p.residual || (p.rs % V == 0 && p.ros % V == 0 && aligned(p.residual, 16) && aligned(p.residual_out, 16)));
    const int ept = p.hidden <= 2048 ? 8 : p.hidden <= 8192 ? 16 : 32;
    const int threads = ((p.hidden + ept - 1) / ept + 31) / 32 * 32;
    const unsigned grid = static_cast<unsigned>(p.rows);
    if (vec) {
        if (ept == 8) norm_kernel<T, V, 8><<<grid, threads, 0, stream>>>(p);
        else if (ept == 16) norm_kernel<T, V, 16><<<grid, threads, 0, stream>>>(p);
        else norm_kernel<T, V, 32><<<grid, threads, 0, stream>>>(p);
    } else {
        if (ept == 8) norm_kernel<T, 1, 8><<<grid, threads, 0, stream>>>(p);
        else if (ept == 16) norm_kernel<T, 1, 16><<<grid, threads, 0, stream>>>(p);
        else norm_kernel<T, 1, 32><<<grid, threads, 0, stream>>>(p);
    }
    return cudaGetLastError();
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
