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
// element.  The kernel is persistent and walks units of kRows rows of one
// (sequence, head), contiguous in the pool, through a ring of shared-memory
// stages: producer warps resolve slots, stage q, k and v as floats and start the
// bulk copy of the unit's rows; the consumers update the rows in the stage and
// read the outputs out; one thread starts the bulk copy back and releases the
// stage once it has been read.  The bytes in flight are thus set by the ring,
// not by registers.  Eight lanes share a row, each taking the 16-byte pieces lane,
// lane + 8, ... of it: a quarter of a warp touches 128 contiguous bytes.
//
// 256 sequences x 32 heads of 128 x 128 fp32 states: 173 us, 6.3 TB/s, 0.92 of the
// copy rate (plain loads and stores by registers, 96 KB in flight an SM: 194 us).
// Other heads (dim x dstate) with states of 0.5 GB: fp32 64 x 64, 64 x 128, 128 x 64,
// 112 x 112 and 120 x 128 0.93 to 0.95, 80 x 96 and 96 x 80 0.90, 72 x 96 0.82, 32 x 32
// 0.36; bf16 128 x 128 and 64 x 128 0.80, 120 x 128 0.76, 112 x 112 0.62, 64 x 64 and
// 128 x 64 0.56, 80 x 96, 96 x 80 and 72 x 96 0.38 to 0.43, 32 x 32 0.17.  A unit costs
// the same however few bytes its rows have, and a dim that is no multiple of 64 has a
// unit of few rows.
#include "ssu_device.cuh"
#include "ssu_hybrid.h"

namespace ssu {

namespace {

constexpr int kLanes = 8;
constexpr int kConsumers = 256;
constexpr int kSlots = kConsumers / kLanes;  // rows in one pass
constexpr int kRows = 64;                    // rows of a unit
constexpr int kProducers = 2;                // warps
constexpr int kThreads = kConsumers + 32 * kProducers;
// Shared memory an SM can give its CTAs, less a margin: two CTAs of up to six
// stages share it.
constexpr int kSmemPerCta = 222 * 1024 / 2 - 1024;
constexpr int kMaxStages = 6;

struct Header {
    int64_t ws;     // destination slot
    float dA;       // exp(log_decay)
    int32_t flags;  // kUnit*
};
enum : int32_t { kUnitValid = 1, kUnitSeeded = 2, kUnitWrite = 4 };

// Layout of a stage: the rows, q, k, v, the header.
struct Ring {
    int tile, stage, stages, units_per_head;
    __host__ __device__ Ring(int n, int size, int dim) {
        tile = kRows * n * size;
        stage = (tile + (2 * kLinattnMaxDim + kRows) * 4 + static_cast<int>(sizeof(Header)) + 127) / 128 * 128;
        stages = (kSmemPerCta - 512) / stage;
        if (stages > kMaxStages) stages = kMaxStages;
        units_per_head = (dim + kRows - 1) / kRows;
    }
    __host__ __device__ int bytes() const { return stages * stage + 16 * stages + static_cast<int>(sizeof(RingExit)); }
};

// A unit's place.
struct UnitAt {
    int64_t b;
    int h, row0, rows;
    __device__ __forceinline__ UnitAt(const LinattnParams &p, int per, int64_t u) {
        const int64_t bh = u / per;
        row0 = static_cast<int>(u - bh * per) * kRows;
        b = bh / p.H;
        h = static_cast<int>(bh - b * p.H);
        rows = min(kRows, p.P - row0);
    }
};

// What a producer needs of a unit, loaded one unit ahead.
struct Operands {
    uint32_t q[kLinattnMaxDim / 32], k[kLinattnMaxDim / 32], v[kRows / 32];
    int64_t rs, ws;
    float g;
    bool ok;
    template <bool WIDE>
    __device__ __forceinline__ void load_rows(const LinattnParams &p, const UnitAt &at, int lane) {
        const int gh = at.h / p.share;
        const int64_t qo = at.b * p.qs[0] + at.h * p.qs[1], ko = at.b * p.ks[0] + gh * p.ks[1];
        const int64_t vo = at.b * p.vs[0] + gh * p.vs[1] + at.row0;
#pragma unroll
        for (int i = 0; i < kLinattnMaxDim / 32; ++i) {
            const int n = lane + 32 * i;
            if (n < p.N) {
                q[i] = load_bits<WIDE>(p.q, qo + n);
                k[i] = load_bits<WIDE>(p.k, ko + n);
            }
        }
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i)
            if (lane + 32 * i < at.rows) v[i] = load_bits<WIDE>(p.v, vo + lane + 32 * i);
    }
    __device__ __forceinline__ void load(const LinattnParams &p, const UnitAt &at, int lane) {
        ok = true;
        rs = ws = 0;
        if (lane == 0) {
            KParams kp{};
            kp.slots = p.slots;
            kp.pad = p.pad;
            kp.status = p.status;
            ok = table_slot(kp, p.rd, at.b, 0, at.b, at.b, &rs);
            ws = rs;
            if (p.wr.entries != nullptr) ok = table_slot(kp, p.wr, at.b, 0, at.b, at.b, &ws) && ok;
            ok = ok && slot_ok(kp, rs) && slot_ok(kp, ws);
        }
        if (p.io_dtype == kF32) load_rows<true>(p, at, lane);
        else load_rows<false>(p, at, lane);
        g = __ldg(p.log_decay + at.h);
    }
};

// Stages unit number k of this CTA; false when the CTA stops.
template <typename TS>
__device__ __forceinline__ bool produce(const LinattnParams &p, const Ring &r, const Operands &op, const UnitAt &at, int k,
                                        unsigned char *smem, uint64_t *full, uint64_t *empty, RingExit *rx, int lane) {
    const int s = k % r.stages, round = k / r.stages;
    if (ring_aborted(rx)) return false;
    if (round > 0 && !mbar_wait_bounded(&empty[s], (round - 1) & 1)) {
        if (lane == 0) {
            flag(p.status, kDevTimeout);
            ring_abort(rx);
        }
        return false;
    }
    unsigned char *st = smem + s * r.stage;
    float *q = reinterpret_cast<float *>(st + r.tile), *kk = q + kLinattnMaxDim, *v = kk + kLinattnMaxDim;
    Header *hd = reinterpret_cast<Header *>(v + kRows);
    int32_t flags = 0;
    if (lane == 0) {
        if (op.ok) {
            flags = kUnitValid;
            if (op.rs != p.pad) flags |= kUnitSeeded;
            if (op.ws != p.pad) flags |= kUnitWrite;
        }
        hd->ws = op.ws;
        hd->dA = expf(op.g);
        hd->flags = flags;
    }
#pragma unroll
    for (int i = 0; i < kLinattnMaxDim / 32; ++i) {
        const int n = lane + 32 * i;
        if (n < p.N) {
            q[n] = bits_to_float(op.q[i], p.io_dtype);
            kk[n] = bits_to_float(op.k[i], p.io_dtype);
        }
    }
#pragma unroll
    for (int i = 0; i < kRows / 32; ++i)
        if (lane + 32 * i < at.rows) v[lane + 32 * i] = bits_to_float(op.v[i], p.io_dtype);
    flags = __shfl_sync(0xffffffffu, flags, 0);
    if (flags & kUnitSeeded) {
        if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(at.rows) * p.N * sizeof(TS);
            const TS *src = static_cast<const TS *>(p.state) + ((op.rs * p.H + at.h) * static_cast<int64_t>(p.P) + at.row0) * p.N;
            mbar_arrive_expect(&full[s], bytes);
            bulk_load(st, src, bytes, &full[s]);
        }
    } else if (lane == 0) {
        mbar_arrive(&full[s]);
    }
    if (lane == 0) ring_note_fill(rx, s, round);
    else mbar_arrive(&full[s]);
    return true;
}

// NC: 16-byte pieces a lane holds of one row.
template <typename TS, int NC>
__global__ void __launch_bounds__(kThreads, 2) linattn_step_kernel(const LinattnParams p, const Ring r, int64_t units) {
    using SC = StateChunk<TS>;
    constexpr int V = SC::kVec;
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + r.stages * r.stage), *empty = full + r.stages;
    RingExit *rx = reinterpret_cast<RingExit *>(empty + r.stages);
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int s = 0; s < r.stages; ++s) {
            mbar_init(&full[s], 32);
            mbar_init(&empty[s], 1);
        }
        ring_init(rx);
    }
    __syncthreads();
    int done = 0;  // units consumed
    if (warp >= kConsumers / 32) {
        const int w = warp - kConsumers / 32, lane = tid & 31;
        const int64_t step = static_cast<int64_t>(kProducers) * gridDim.x;
        int64_t u = blockIdx.x + static_cast<int64_t>(w) * gridDim.x;
        Operands now, next;
        if (u < units) now.load(p, UnitAt(p, r.units_per_head, u), lane);
        for (int k = w; u < units; k += kProducers, u += step) {
            if (u + step < units) next.load(p, UnitAt(p, r.units_per_head, u + step), lane);
            if (!produce<TS>(p, r, now, UnitAt(p, r.units_per_head, u), k, smem, full, empty, rx, lane)) break;
            now = next;
        }
    } else {
        const int lane = tid % kLanes, r0 = tid / kLanes, pieces = p.N / V;
        int prev = -1;
        for (int64_t u = blockIdx.x; u < units; u += gridDim.x, ++done) {
            const int s = done % r.stages;
            const bool ok = mbar_wait_bounded(&full[s], (done / r.stages) & 1);
            if (barrier_or(1, kConsumers, !ok)) {  // a wait gave up: every consumer stops here
                if (tid == 0) {
                    flag(p.status, kDevTimeout);
                    ring_abort(rx);
                    bulk_wait_all();
                }
                break;
            }
            unsigned char *st = smem + s * r.stage;
            const float *q = reinterpret_cast<const float *>(st + r.tile), *k = q + kLinattnMaxDim, *v = k + kLinattnMaxDim;
            const Header hd = *reinterpret_cast<const Header *>(v + kRows);
            const UnitAt at(p, r.units_per_head, u);
            if (hd.flags & kUnitValid) {
                float qv[NC * V], kv[NC * V];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const int n = (lane + kLanes * c) * V;
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        float4 f = make_float4(0.f, 0.f, 0.f, 0.f), e = f;
                        if (lane + kLanes * c < pieces) {
                            f = *reinterpret_cast<const float4 *>(q + n + i);
                            e = *reinterpret_cast<const float4 *>(k + n + i);
                        }
                        qv[c * V + i] = f.x, qv[c * V + i + 1] = f.y, qv[c * V + i + 2] = f.z, qv[c * V + i + 3] = f.w;
                        kv[c * V + i] = e.x, kv[c * V + i + 1] = e.y, kv[c * V + i + 2] = e.z, kv[c * V + i + 3] = e.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < kRows / kSlots; ++i) {
                    const int row = r0 + i * kSlots;
                    const bool live = row < at.rows;
                    TS *mine = reinterpret_cast<TS *>(st) + row * p.N;
                    const float vr = live ? v[row] : 0.f;
                    float sum = 0.f;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        if (!live || lane + kLanes * c >= pieces) continue;
                        uint4 *piece = reinterpret_cast<uint4 *>(mine + (lane + kLanes * c) * V);
                        float x[V];
                        SC::unpack(hd.flags & kUnitSeeded ? *piece : make_uint4(0u, 0u, 0u, 0u), x);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            x[e] = fmaf(x[e], hd.dA, vr * kv[c * V + e]);
                            sum = fmaf(x[e], qv[c * V + e], sum);
                        }
                        *piece = SC::pack(x);
                    }
                    sum = row_sum<kLanes>(sum);
                    if (lane == 0 && live)
                        store_small(p.out, at.b * p.os[0] + at.h * p.os[1] + at.row0 + row, p.io_dtype, p.scale * sum);
                }
            }
            fence_proxy_async_smem();
            named_barrier(1, kConsumers);
            if (tid == 0) {
                if ((hd.flags & kUnitValid) && (hd.flags & kUnitWrite)) {
                    TS *dst = static_cast<TS *>(p.state) + ((hd.ws * p.H + at.h) * static_cast<int64_t>(p.P) + at.row0) * p.N;
                    bulk_store(dst, st, static_cast<uint32_t>(at.rows) * p.N * sizeof(TS));
                }
                bulk_commit();
                // the previous unit's rows have been read out by their copy:
                // its stage may be refilled
                if (prev >= 0) {
                    bulk_wait_read<1>();
                    mbar_arrive(&empty[prev]);
                }
            }
            prev = s;
        }
        if (tid == 0) bulk_wait_all();
    }
    __syncthreads();
    if (tid == 0) ring_drain(rx, full, r.stages, done, kWaitCycles, p.status);
}

template <typename TS, int NC>
cudaError_t launch_nc(const LinattnParams &p, cudaStream_t stream) {
    static int resident[64];  // CTAs the device holds, by device
    const Ring r(p.N, sizeof(TS), p.P);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) dev = 0;
    int n = __atomic_load_n(&resident[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        int sms = 0, per = 0;
        if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
        if ((e = cudaFuncSetAttribute(linattn_step_kernel<TS, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerCta)) !=
            cudaSuccess)
            return e;
        if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, linattn_step_kernel<TS, NC>, kThreads, kSmemPerCta)) !=
            cudaSuccess)
            return e;
        if (per <= 0) return cudaErrorInvalidConfiguration;
        n = sms * per;
        __atomic_store_n(&resident[dev], n, __ATOMIC_RELAXED);
    }
    const int64_t units = p.rows * p.H * r.units_per_head;
    const int64_t grid = units < n ? units : n;
    linattn_step_kernel<TS, NC><<<static_cast<unsigned>(grid), kThreads, r.bytes(), stream>>>(p, r, units);
    return cudaGetLastError();
}

template <typename TS>
cudaError_t launch_step_t(const LinattnParams &p, cudaStream_t stream) {
    const int per = StateChunk<TS>::kVec * kLanes;
    switch ((p.N + per - 1) / per) {
    case 1: return launch_nc<TS, 1>(p, stream);
    case 2: return launch_nc<TS, 2>(p, stream);
    case 3:
        if constexpr (sizeof(TS) == 4) return launch_nc<TS, 3>(p, stream);
        break;
    case 4:
        if constexpr (sizeof(TS) == 4) return launch_nc<TS, 4>(p, stream);
        break;
    }
    return cudaErrorInvalidValue;
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
