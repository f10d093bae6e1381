// ssu_linattn_prefill.cu -- linear attention with a decay for each head over
// packed prompts: the recurrence itself, token by token.
//     S_t = exp(log_decay[h]) S_{t-1} + v_t k_t^T,   out_t = scale S_t q_t
// One CTA takes 32 dim rows of one (sequence, head) and carries them in fp32
// registers, eight lanes a row; q, k and v of kBlock tokens are staged at a
// time.
#include "ssu_device.cuh"
#include "ssu_hybrid.h"

namespace ssu {

namespace {

constexpr int kLanes = 8;
constexpr int kThreads = 256;
constexpr int kRows = kThreads / kLanes;
constexpr int kBlock = 16;
constexpr int kPer = kLinattnMaxDim / kLanes;  // columns lane * kPer ... of a row

__device__ __forceinline__ float load_state(const void *s, int dtype, int64_t i) {
    if (dtype == kF32) return static_cast<const float *>(s)[i];
    return bits_to_float(static_cast<const unsigned short *>(s)[i], dtype);
}
__device__ __forceinline__ float load_io(const void *s, int dtype, int64_t i) {
    return bits_to_float(load_bits<false>(s, i), dtype);
}

__global__ void __launch_bounds__(kThreads) linattn_prefill_kernel(const LinattnParams p, int tiles) {
    __shared__ __align__(16) float qs[kBlock][kLinattnMaxDim], ks[kBlock][kLinattnMaxDim], vs[kBlock][kRows];
    __shared__ int64_t slot[2];
    const int tid = threadIdx.x, lane = tid % kLanes, r = tid / kLanes;
    const int tile = blockIdx.x % tiles;
    const int64_t bh = blockIdx.x / tiles;
    const int h = static_cast<int>(bh % p.H);
    const int64_t b = bh / p.H;
    const int g = h / p.share;
    const int64_t t0 = load_index(p.cu, b, p.meta_is_i64), t1 = load_index(p.cu, b + 1, p.meta_is_i64);
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
        if (t0 < 0 || t1 < t0 || t1 > p.rows) {
            flag(p.status, kDevBadSeqlen);
            ok = false;
        }
        slot[0] = ok ? (rs == p.pad ? -1 : rs) : -2;
        slot[1] = ws == p.pad ? -1 : ws;
    }
    __syncthreads();
    const int64_t rs = slot[0], ws = slot[1];
    if (rs == -2) return;
    const int row = tile * kRows + r;
    const float dA = expf(__ldg(p.log_decay + h));
    float s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = lane * kPer + i;
        s[i] = 0.f;
        if (rs >= 0 && row < p.P && n < p.N) s[i] = load_state(p.state, p.state_dtype, ((rs * p.H + h) * p.P + row) * p.N + n);
    }
    for (int64_t t = t0; t < t1; t += kBlock) {
        const int m = t1 - t < kBlock ? static_cast<int>(t1 - t) : kBlock;
        __syncthreads();
        for (int i = tid; i < kBlock * kLinattnMaxDim; i += kThreads) {
            const int j = i / kLinattnMaxDim, n = i % kLinattnMaxDim;
            const bool in = j < m && n < p.N;
            qs[j][n] = in ? load_io(p.q, p.io_dtype, (t + j) * p.qs[0] + h * p.qs[1] + n) : 0.f;
            ks[j][n] = in ? load_io(p.k, p.io_dtype, (t + j) * p.ks[0] + g * p.ks[1] + n) : 0.f;
        }
        for (int i = tid; i < kBlock * kRows; i += kThreads) {
            const int j = i / kRows, q = tile * kRows + i % kRows;
            vs[j][i % kRows] = j < m && q < p.P ? load_io(p.v, p.io_dtype, (t + j) * p.vs[0] + g * p.vs[1] + q) : 0.f;
        }
        __syncthreads();
        for (int j = 0; j < m; ++j) {
            const float v = vs[j][r];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                s[i] = fmaf(s[i], dA, v * ks[j][lane * kPer + i]);
                sum = fmaf(s[i], qs[j][lane * kPer + i], sum);
            }
            sum = row_sum<kLanes>(sum);
            if (lane == 0 && row < p.P) store_small(p.out, (t + j) * p.os[0] + h * p.os[1] + row, p.io_dtype, p.scale * sum);
        }
    }
    if (ws >= 0 && row < p.P) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int n = lane * kPer + i;
            if (n < p.N) store_small(p.state, ((ws * p.H + h) * p.P + row) * p.N + n, p.state_dtype, s[i]);
        }
    }
}

}  // namespace

cudaError_t launch_linattn_prefill(const LinattnParams &p, cudaStream_t stream) {
    const int tiles = (p.P + kRows - 1) / kRows;
    linattn_prefill_kernel<<<static_cast<unsigned>(p.nseq * p.H * tiles), kThreads, 0, stream>>>(p, tiles);
    return cudaGetLastError();
}

}  // namespace ssu
