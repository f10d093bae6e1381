// ssu_linattn_step.cu -- linear attention with a decay for each head, one
// token per sequence (the recurrent form).
//
// Sequence b, head h of key/value head g = h / share, S = its slot's state
// [dim, dstate]:
//     S <- exp(log_decay[h]) S + v k^T,   out = scale S q
// The state is carried in fp32 between the read and the write and rounded
// once, to nearest even, into the pool's type.
//
// HBM-bound: every state byte is read once and written once, two FMAs per
// element.  One CTA takes kRows rows of one (sequence, head); eight lanes share
// a row, each holding the 16-byte pieces lane, lane + 8, ... of it, and a
// thread has all its pieces of kRows / 32 rows in flight at once.
#include "ssu_device.cuh"
#include "ssu_hybrid.h"

namespace ssu {

namespace {

constexpr int kLanes = 8;
constexpr int kThreads = 256;
constexpr int kSlots = kThreads / kLanes;  // rows in one pass
constexpr int kPasses = 2;
constexpr int kRows = kSlots * kPasses;

// NC: 16-byte pieces a lane holds of one row.
template <typename TS, int NC>
__global__ void __launch_bounds__(kThreads) linattn_step_kernel(const LinattnParams p, int tiles) {
    using SC = StateChunk<TS>;
    constexpr int V = SC::kVec;
    __shared__ __align__(16) float qs[kLinattnMaxDim], ks[kLinattnMaxDim];
    __shared__ int64_t slot[2];
    const int tid = threadIdx.x, lane = tid % kLanes, r0 = tid / kLanes;
    const int tile = blockIdx.x % tiles;
    const int64_t bh = blockIdx.x / tiles;
    const int h = static_cast<int>(bh % p.H);
    const int64_t b = bh / p.H;
    const int g = h / p.share;
    if (tid == 0) {
        int64_t rs = 0, ws = 0;
        KParams kp{};
        kp.slots = p.slots;
        kp.pad = p.pad;
        kp.status = p.status;
        bool ok = table_slot(kp, p.rd, b, 0, b, b, &rs);
        ws = rs;
        if (p.wr.entries != nullptr) ok = table_slot(kp, p.wr, b, 0, b, b, &ws) && ok;
        ok = ok && slot_ok(kp, rs) && slot_ok(kp, ws);
        slot[0] = ok ? (rs == p.pad ? -1 : rs) : -2;
        slot[1] = ws == p.pad ? -1 : ws;
    }
    // q and k of the token, as floats (their rows may have any alignment)
    for (int n = tid; n < p.N; n += kThreads) {
        const int64_t qo = b * p.qs[0] + h * p.qs[1] + n, ko = b * p.ks[0] + g * p.ks[1] + n;
        if (p.io_dtype == kF32) {
            qs[n] = __uint_as_float(load_bits<true>(p.q, qo));
            ks[n] = __uint_as_float(load_bits<true>(p.k, ko));
        } else {
            qs[n] = bits_to_float(load_bits<false>(p.q, qo), p.io_dtype);
            ks[n] = bits_to_float(load_bits<false>(p.k, ko), p.io_dtype);
        }
    }
    __syncthreads();
    const int64_t rs = slot[0], ws = slot[1];
    if (rs == -2) return;  // flagged: nothing of this unit is written
    const int pieces = p.N / V;
    uint4 raw[kPasses][NC];
    float v[kPasses];
    const TS *src = static_cast<const TS *>(p.state) + (rs * p.H + h) * static_cast<int64_t>(p.P) * p.N;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int row = tile * kRows + r0 + i * kSlots;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            raw[i][c] = make_uint4(0u, 0u, 0u, 0u);
            if (rs >= 0 && row < p.P && lane + kLanes * c < pieces)
                raw[i][c] = ld_stream(src + static_cast<int64_t>(row) * p.N + (lane + kLanes * c) * V);
        }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int row = tile * kRows + r0 + i * kSlots;
        v[i] = 0.f;
        if (row < p.P) {
            const int64_t vo = b * p.vs[0] + g * p.vs[1] + row;
            v[i] = p.io_dtype == kF32 ? __uint_as_float(load_bits<true>(p.v, vo)) : bits_to_float(load_bits<false>(p.v, vo), p.io_dtype);
        }
    }
    const float dA = expf(__ldg(p.log_decay + h));
    float qv[NC * V], kv[NC * V];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int n = (lane + kLanes * c) * V;
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f), e = f;
            if (lane + kLanes * c < pieces) {
                f = *reinterpret_cast<const float4 *>(qs + n + i);
                e = *reinterpret_cast<const float4 *>(ks + n + i);
            }
            qv[c * V + i] = f.x, qv[c * V + i + 1] = f.y, qv[c * V + i + 2] = f.z, qv[c * V + i + 3] = f.w;
            kv[c * V + i] = e.x, kv[c * V + i + 1] = e.y, kv[c * V + i + 2] = e.z, kv[c * V + i + 3] = e.w;
        }
    }
    TS *dst = static_cast<TS *>(p.state) + (ws * p.H + h) * static_cast<int64_t>(p.P) * p.N;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int row = tile * kRows + r0 + i * kSlots;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float s[V];
            SC::unpack(raw[i][c], s);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[e] = fmaf(s[e], dA, v[i] * kv[c * V + e]);
                sum = fmaf(s[e], qv[c * V + e], sum);
            }
            if (ws >= 0 && row < p.P && lane + kLanes * c < pieces)
                st_stream(dst + static_cast<int64_t>(row) * p.N + (lane + kLanes * c) * V, SC::pack(s));
        }
        sum = row_sum<kLanes>(sum);
        if (lane == 0 && row < p.P)
            store_small(p.out, b * p.os[0] + h * p.os[1] + row, p.io_dtype, p.scale * sum);
    }
}

template <typename TS>
cudaError_t launch_step_t(const LinattnParams &p, cudaStream_t stream) {
    const int per = StateChunk<TS>::kVec * kLanes;
    const int nc = (p.N + per - 1) / per;
    const int tiles = (p.P + kRows - 1) / kRows;
    const unsigned grid = static_cast<unsigned>(p.rows * p.H * tiles);
    switch (nc) {
    case 1: linattn_step_kernel<TS, 1><<<grid, kThreads, 0, stream>>>(p, tiles); break;
    case 2: linattn_step_kernel<TS, 2><<<grid, kThreads, 0, stream>>>(p, tiles); break;
    case 3:
        if constexpr (sizeof(TS) == 4) linattn_step_kernel<TS, 3><<<grid, kThreads, 0, stream>>>(p, tiles);
        break;
    case 4:
        if constexpr (sizeof(TS) == 4) linattn_step_kernel<TS, 4><<<grid, kThreads, 0, stream>>>(p, tiles);
        break;
    default: return cudaErrorInvalidValue;
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_step(const LinattnParams &p, cudaStream_t stream) {
    switch (p.state_dtype) {
    case kF32: return launch_step_t<float>(p, stream);
    case kF16: return launch_step_t<__half>(p, stream);
    case kBF16: return launch_step_t<__nv_bfloat16>(p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace ssu
