// ssu_linattn_prefill.cu -- linear attention with a decay for each head over
// packed prompts: the chunked form on the 5th-generation tensor cores.
//
// The recurrence S_t = l S_{t-1} + v_t k_t^T, out_t = scale S_t q_t, l =
// e^log_decay[h], over a chunk of n <= 128 tokens (i, j within it) with S the
// state that enters it:
//     out_i = scale (l^(i+1) S q_i + sum_{j<=i} l^(i-j) (q_i . k_j) v_j)
//     S'    = l^n S + sum_j l^(n-1-j) v_j k_j^T
// A work unit is one piece of a sequence (all of it, or an equal part of a long
// one) for one head; a CTA walks its chunks and carries S in registers.
//
// Four products a chunk, tcgen05.mma with fp32 accumulators in tensor memory:
//   scores   [i, j]    = Q K^T             Q, K from shared memory, as loaded
//   entering [p, i]    = S Q^T             S as a high and a low part, from tensor memory
//   inside   [p, i]    = V^T P^T           P = scores decayed and masked, rounded once
//   growth   [p, n]    = (V decayed)^T K   the decayed V in three parts (bf16) or two
//                                          (fp16), from tensor memory
// Outputs, states and the decayed values thus share lanes: lane p of tensor
// memory belongs to value dim p, so l^n S + growth, the split of S into parts
// and the transposition of V (read by columns from shared memory) stay within a
// thread.  The decay of the entering state is applied to the product, in fp32.
// Rounding: P to the io type (2^-8 bf16, 2^-11 fp16, as the output itself); S
// where it meets Q to two parts (2^-16, 2^-22); the decayed V to three parts
// (2^-24) or two (2^-22), so that fp32 states keep fp32 accuracy.  fp16 parts are
// scaled by powers of two (per state row, score row and value tile), so neither
// overflow nor the subnormals cost accuracy.
//
// Warps: 0-3 turn scores into P and store outputs (thread = score row, then
// value dim); 4-7 own S (thread = value dim), split it, and decay V; 8 issues
// the products; 9 finds the units and loads Q, K, V (tiled copies, two stages);
// 10 and 11 only complete the third group, whose registers the others take.
#include <cuda.h>

#include "ssu_hybrid.h"
#include "ssu_tcgen05.cuh"

namespace ssu {

namespace {

constexpr int kC = 128;       // tokens of a chunk
constexpr int kPanel = 16384;  // 128 rows of 128 bytes
constexpr int kThreads = 384;
constexpr int kGroup = 128;   // threads of one of the two groups of warps
constexpr int kQuarter = 32;  // tokens whose decayed V is handed over at a time

// Tensor-memory columns.  The decayed V goes where the parts of S were, once
// the entering product has read them.
constexpr uint32_t kColScore = 0, kColOut = 128, kColGrowth = 256, kColState = 384;
constexpr uint32_t kRing = 48;  // columns of one quarter: up to 3 parts of 16

struct Unit {
    int64_t t0;      // first token row
    int64_t src;     // state entering: pool slot or kZero
    int64_t dst;     // state leaving: pool slot or kNone
    int32_t len;     // tokens; -1: no more units
    int32_t h;
};
constexpr int64_t kZero = -1, kNone = -1;

enum : int {
    kFull0, kFull1,    // a stage's Q, K, V have landed
    kFree0, kFree1,    // ... and are done with
    kUnitFull0, kUnitFull1, kUnitFree0, kUnitFree1,
    kScore,            // the scores are there
    kStateFull,        // the parts of S are there
    kEnter,            // the entering product is there (and the parts of S are read)
    kPFull,            // P is there; the scores and the entering product are read
    kInside,           // the inside product is there (and P is read)
    kOutFree,          // ... and read
    kTail,             // a partial chunk's K and V rows past its end are zeros
    kVFull0, kVFull1, kVFree0, kVFree1,
    kGrowth,
    kSyncA, kSyncB,
    kFinal,
    kBars
};

template <int DK>
struct Layout {
    static constexpr int kQBytes = DK / 64 * kPanel;
    static constexpr int kKBytes = kQBytes;
    static constexpr int kVBytes = 2 * kPanel;
    static constexpr int kStage = kQBytes + kKBytes + kVBytes;
    static constexpr int kP = 2 * kStage;              // P: two panels
    static constexpr int kBar = kP + 2 * kPanel;
    static constexpr int kUnits = kBar + 8 * kBars;     // Unit[2]
    static constexpr int kTabA = (kUnits + 2 * static_cast<int>(sizeof(Unit)) + 15) / 16 * 16;  // scale l^(i+1), 128 floats
    static constexpr int kTabB = kTabA + 128 * 4;       // l^(127-j), j < 128, then a quarter of zeros
    static constexpr int kRowScale = kTabB + (128 + 32) * 4;  // fp16: of the state rows, then of the score rows
    static constexpr int kMax = kRowScale + 256 * 4;    // fp16: per warp
    static constexpr int kMisc = kMax + 16;             // tensor-memory address, abort
    static constexpr int kBytes = kMisc + 16;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap q, k, v;
};

// A barrier of one group of warps, its waits bounded like every other.
__device__ __forceinline__ bool group_sync(uint64_t *bar, int &phase) {
    mbar_arrive(bar);
    const bool ok = mbar_wait_bounded(bar, phase & 1);
    ++phase;
    return ok;
}

// Two floats as the io type, and what the pair stands for.
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
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    if constexpr (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// Gives up (N below 168) or takes registers; every warp of a group of four
// calls it with the same N.
template <int N>
__device__ __forceinline__ void registers() {
    if constexpr (N < 168) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Finds unit u of the call: the sequence's bounds and slots.  False (and
// flagged) when it is to be skipped.
__device__ __forceinline__ bool find_unit(const LinattnParams &p, int64_t u, Unit &out) {
    const int64_t b = u / p.H;
    out.h = static_cast<int>(u - b * p.H);
    const int64_t t0 = load_index(p.cu, b, p.meta_is_i64), t1 = load_index(p.cu, b + 1, p.meta_is_i64);
    KParams kp{};
    kp.slots = p.slots;
    kp.pad = p.pad;
    kp.status = p.status;
    int64_t rs = 0, ws = 0;
    bool ok = table_slot(kp, p.rd, b, 0, b, b, &rs);
    ws = rs;
    if (p.wr.entries != nullptr) ok = table_slot(kp, p.wr, b, 0, b, b, &ws) && ok;
    ok = ok && slot_ok(kp, rs) && slot_ok(kp, ws);
    if (t0 < 0 || t1 < t0 || t1 > p.rows) {
        flag(p.status, kDevBadSeqlen);
        ok = false;
    }
    out.t0 = t0;
    out.len = static_cast<int>(t1 - t0);
    out.src = rs == p.pad ? kZero : rs;
    out.dst = ws == p.pad ? kNone : ws;
    return ok;
}

template <int DK, bool BF>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_prefill_kernel(const LinattnParams p, const __grid_constant__ Maps maps, int64_t units) {
    using LY = Layout<DK>;
    constexpr int kParts = BF ? 3 : 2;  // parts of the decayed V
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + LY::kBar);
    Unit *ring = reinterpret_cast<Unit *>(smem + LY::kUnits);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + LY::kMisc);
    volatile uint32_t *abort_flag = misc + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            int n = 1;
            if (i == kFree0 || i == kFree1) n = 1 + kGroup;
            if (i == kUnitFree0 || i == kUnitFree1) n = 1 + 2 * kGroup;
            if (i == kStateFull || i == kPFull || i == kOutFree || i == kTail || i == kVFull0 ||
                i == kVFull1 || i == kSyncA || i == kSyncB)
                n = kGroup;
            mbar_init(&bars[i], n);
        }
        *abort_flag = 0;
    }
    if (p.P <= 64) {
        // values of dims 64 .. 127 do not exist: their panels stay zero
        for (int i = tid; i < 2 * kPanel / 16; i += kThreads)
            *reinterpret_cast<uint4 *>(smem + (i / (kPanel / 16)) * LY::kStage + LY::kQBytes + LY::kKBytes + kPanel +
                                       (i % (kPanel / 16)) * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (warp == 8) tmem_alloc512(misc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    bool ok = true;

    // The launch gives every thread 168 registers (3 groups x 128 x 168 in
    // all); the two compute groups take 216 each, 72 are left for the third.
    if (warp == 9) {
        registers<72>();
        // ---------------- units and loads ----------------
        if (lane == 0) {
            int nu = 0, ch = 0;  // units published, chunks loaded
            const int vpanels = p.P > 64 ? 2 : 1;
            for (int64_t u = blockIdx.x;; u += gridDim.x) {
                Unit un;
                const bool end = u >= units;
                if (end) un.len = -1;
                else if (!find_unit(p, u, un)) continue;
                if (nu >= 2 && !(ok = mbar_wait_bounded(&bars[kUnitFree0 + (nu & 1)], ((nu >> 1) - 1) & 1))) break;
                ring[nu & 1] = un;
                mbar_arrive(&bars[kUnitFull0 + (nu & 1)]);
                ++nu;
                if (end) break;
                const int g = un.h / p.share;
                for (int c = 0; c < un.len; c += kC, ++ch) {
                    const int s = ch & 1;
                    if (ch >= 2 && !(ok = mbar_wait_bounded(&bars[kFree0 + s], ((ch >> 1) - 1) & 1))) break;
                    if (*abort_flag) ok = false;
                    if (!ok) break;
                    unsigned char *st = smem + s * LY::kStage;
                    mbar_arrive_expect(&bars[kFull0 + s], LY::kQBytes + LY::kKBytes + vpanels * kPanel);
                    const int row = static_cast<int>(un.t0) + c;
                    for (int i = 0; i < DK / 64; ++i) {
                        tma_load_3d(st + i * kPanel, &maps.q, 64 * i, un.h, row, &bars[kFull0 + s]);
                        tma_load_3d(st + LY::kQBytes + i * kPanel, &maps.k, 64 * i, g, row, &bars[kFull0 + s]);
                    }
                    for (int i = 0; i < vpanels; ++i)
                        tma_load_3d(st + LY::kQBytes + LY::kKBytes + i * kPanel, &maps.v, 64 * i, g, row, &bars[kFull0 + s]);
                }
                if (!ok) break;
            }
            if (!ok) {
                flag(p.status, kDevTimeout);
                *abort_flag = 1;
            }
            // what was loaded has landed before the CTA retires
            for (int k = ch > 2 ? ch - 2 : 0; k < ch; ++k) mbar_wait_bounded(&bars[kFull0 + (k & 1)], (k >> 1) & 1);
        }
        __syncwarp();
    } else if (warp == 8) {
        registers<72>();
        // ---------------- products (one thread) ----------------
        if (lane == 0) {
            constexpr int bf = BF ? 1 : 0;
            constexpr uint32_t kIdScore = idesc_f16(128, 128, 0, 0, bf), kIdEnter = idesc_f16(128, 128, 0, 0, bf);
            constexpr uint32_t kIdInside = idesc_f16(128, 128, 1, 0, bf), kIdGrowth = idesc_f16(128, DK, 0, 1, bf);
            // Descriptors differ by constants: their address field counts 16 bytes.
            const uint32_t sQ = smem_addr(smem);
            const uint64_t dQ = desc_k_sw128(sQ), dK = desc_k_sw128(sQ + LY::kQBytes);
            const uint64_t dV = desc_mn_sw128(sQ + LY::kQBytes + LY::kKBytes, kPanel);
            const uint64_t dP = desc_k_sw128(smem_addr(smem + LY::kP));
            const uint64_t kToMn = desc_mn_sw128(0, kPanel) - desc_k_sw128(0);  // the same K read along its tokens
            constexpr auto along_k = [](int k) { return static_cast<uint64_t>(((k / 4) * kPanel + (k % 4) * 32) >> 4); };
            constexpr auto along_mn = [](int k) { return static_cast<uint64_t>((k * 2048) >> 4); };
            const auto stage = [](int s) { return static_cast<uint64_t>(s * (LY::kStage >> 4)); };
            const auto scores = [&](int s) {
                const uint64_t q = dQ + stage(s), k0 = dK + stage(s);
#pragma unroll
                for (int k = 0; k < DK / 16; ++k)
                    mma(tmem + kColScore, q + along_k(k), k0 + along_k(k), kIdScore, k > 0);
                mma_commit(&bars[kScore]);
            };
            int nu = 0, ch = 0, tails = 0, quarters = 0;
            for (;;) {
                if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
                const int len = ring[nu & 1].len;
                mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
                ++nu;
                if (len < 0) break;
                for (int c = 0; c < len; c += kC, ++ch) {
                    const int s = ch & 1, n = min(kC, len - c), steps = (n + 15) / 16;
                    const uint64_t dQs = dQ + stage(s), dVs = dV + stage(s);
                    if (c == 0) {
                        if (!(ok = mbar_wait_bounded(&bars[kFull0 + s], (ch >> 1) & 1))) break;
                        tc_fence_after();
                        scores(s);
                    }
                    if (!(ok = mbar_wait_bounded(&bars[kStateFull], ch & 1))) break;
                    if (ch > 0 && !(ok = mbar_wait_bounded(&bars[kOutFree], (ch - 1) & 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int part = 0; part < 2; ++part)
#pragma unroll
                        for (int k = 0; k < DK / 16; ++k)
                            mma_ts(tmem + kColOut, tmem + kColState + part * (DK / 2) + 8 * k, dQs + along_k(k), kIdEnter,
                                   part > 0 || k > 0);
                    mma_commit(&bars[kEnter]);
                    if (n < kC && !(ok = mbar_wait_bounded(&bars[kTail], tails++ & 1))) break;
                    if (!(ok = mbar_wait_bounded(&bars[kPFull], ch & 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < steps) mma(tmem + kColOut, dVs + along_mn(k), dP + along_k(k), kIdInside, k > 0);
                    mma_commit(&bars[kInside]);
                    // the next chunk's scores, ahead of this one's growth
                    if (c + kC < len) {
                        if (!(ok = mbar_wait_bounded(&bars[kFull0 + (s ^ 1)], ((ch + 1) >> 1) & 1))) break;
                        tc_fence_after();
                        scores(s ^ 1);
                    }
                    const uint64_t dKn = dK + stage(s) + kToMn;
#pragma unroll
                    for (int qd = 0; qd < 4; ++qd) {
                        if (qd * kQuarter >= n) break;
                        const int r = quarters & 1;
                        if (!(ok = mbar_wait_bounded(&bars[kVFull0 + r], (quarters >> 1) & 1))) break;
                        ++quarters;
                        tc_fence_after();
#pragma unroll
                        for (int k = 2 * qd; k < 2 * qd + 2; ++k)
#pragma unroll
                            for (int part = 0; part < kParts; ++part)
                                if (k < steps)
                                    mma_ts(tmem + kColGrowth, tmem + kColState + r * kRing + part * 16 + 8 * (k & 1),
                                           dKn + along_mn(k), kIdGrowth, k > 0 || part > 0);
                        mma_commit(&bars[kVFree0 + r]);
                    }
                    if (!ok) break;
                    mma_commit(&bars[kGrowth]);
                    mma_commit(&bars[kFree0 + s]);
                }
                if (!ok) break;
            }
            if (!ok) {
                flag(p.status, kDevTimeout);
                *abort_flag = 1;
            }
            // every product issued has completed before tensor memory is freed
            mma_commit(&bars[kFinal]);
            mbar_wait_bounded(&bars[kFinal], 0);
        }
        __syncwarp();
    } else if (warp >= 10) {
        registers<72>();
    } else if (warp < 4) {
        registers<216>();
        // ---------------- P and the outputs ----------------
        const int row = tid;  // score row i; later value dim
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        float *tab = reinterpret_cast<float *>(smem + LY::kTabA);
        float *row_scale = reinterpret_cast<float *>(smem + LY::kRowScale);
        int nu = 0, ch = 0, ph = 0;
        for (;;) {
            if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
            const Unit un = ring[nu & 1];
            mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
            ++nu;
            if (un.len < 0) break;
            const float g = fmaxf(__ldg(p.log_decay + un.h), -1e30f);  // 0 * -inf is no power
            const float g2 = g * 1.4426950408889634f;
            // the previous unit's table is no longer read (a thread that is
            // here has stored its last output, the others are past theirs
            // once all have met)
            if (!(ok = group_sync(&bars[kSyncA], ph))) break;
            tab[row] = p.scale * expf(g * static_cast<float>(row + 1));
            float fall[32];  // l^(31 - jj): from a column of a block to the block's last
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) fall[jj] = ex2(g2 * static_cast<float>(31 - jj));
            if (!(ok = group_sync(&bars[kSyncA], ph))) break;
            unsigned short *out = static_cast<unsigned short *>(p.out) + un.h * p.os[1];
            for (int c = 0; c < un.len; c += kC, ++ch) {
                const int n = min(kC, un.len - c);
                if (!(ok = mbar_wait_bounded(&bars[kScore], ch & 1))) break;
                tc_fence_after();
                // row i of P: l^(i-j) score for j <= i.  A block of 32 columns
                // before the warp's rows factors through its last column, both
                // powers at most 1; the block on the diagonal takes one power
                // a score.
                uint32_t pr[64];
                float mx = 0.f;
                float pv[BF ? 1 : 128];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b <= warp) {
                        uint32_t r[32];
                        tmem_ld32(tmem + lanes + kColScore + 32 * b, r);
                        tmem_wait_ld();
                        float e[32];
                        if (b < warp) {
                            const float f = ex2(g2 * static_cast<float>(row - 32 * b - 31));
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj) e[jj] = __uint_as_float(r[jj]) * (f * fall[jj]);
                        } else {
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj) {
                                const float w = ex2(g2 * static_cast<float>(max(lane - jj, 0)));
                                e[jj] = jj <= lane ? __uint_as_float(r[jj]) * w : 0.f;
                            }
                        }
                        if constexpr (BF) {
#pragma unroll
                            for (int jj = 0; jj < 16; ++jj) pr[16 * b + jj] = pack2<BF>(e[2 * jj], e[2 * jj + 1]);
                        } else {
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj) {
                                pv[(32 * b + jj) % (BF ? 1 : 128)] = e[jj];
                                mx = fmaxf(mx, fabsf(e[jj]));
                            }
                        }
                    } else {
#pragma unroll
                        for (int jj = 0; jj < 16; ++jj) pr[16 * b + jj] = 0u;
                        if constexpr (!BF) {
#pragma unroll
                            for (int jj = 0; jj < 32; ++jj) pv[(32 * b + jj) % (BF ? 1 : 128)] = 0.f;
                        }
                    }
                }
                if constexpr (!BF) {
                    const int k = fp16_scale_exp(mx);
                    const float sc = pow2i(k);
#pragma unroll
                    for (int jj = 0; jj < 64; ++jj)
                        pr[jj] = pack2<BF>(pv[(2 * jj) % (BF ? 1 : 128)] * sc, pv[(2 * jj + 1) % (BF ? 1 : 128)] * sc);
                    row_scale[128 + row] = p.scale * pow2i(-k);
                }
                unsigned char *prow = smem + LY::kP + row * 128;
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    *reinterpret_cast<uint4 *>(prow + (j / 8) * kPanel + (((j % 8) ^ (row & 7)) * 16)) =
                        make_uint4(pr[4 * j], pr[4 * j + 1], pr[4 * j + 2], pr[4 * j + 3]);
                fence_proxy_async_smem();
                // what the entering state contributes
                if (!(ok = mbar_wait_bounded(&bars[kEnter], ch & 1))) break;
                tc_fence_after();
                float hold[128];
                const float back = BF ? 1.f : row_scale[row];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kColOut + 32 * b, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int jj = 0; jj < 32; jj += 4) {
                        const float4 t = *reinterpret_cast<const float4 *>(tab + 32 * b + jj);
                        hold[32 * b + jj] = __uint_as_float(r[jj]) * back * t.x;
                        hold[32 * b + jj + 1] = __uint_as_float(r[jj + 1]) * back * t.y;
                        hold[32 * b + jj + 2] = __uint_as_float(r[jj + 2]) * back * t.z;
                        hold[32 * b + jj + 3] = __uint_as_float(r[jj + 3]) * back * t.w;
                    }
                }
                tc_fence_before();
                mbar_arrive(&bars[kPFull]);
                if (!(ok = mbar_wait_bounded(&bars[kInside], ch & 1))) break;
                // (fp16) the other rows' scales, by their own arrivals
                if (!BF && !(ok = mbar_wait_bounded(&bars[kPFull], ch & 1))) break;
                tc_fence_after();
                // outputs [token][value dim] in P's place, then 16 bytes a
                // store along each token's row
                unsigned short *stage = reinterpret_cast<unsigned short *>(smem + LY::kP) + row;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kColOut + 32 * b, r);
                    tmem_wait_ld();
                    if (b == 3) {
                        tc_fence_before();
                        mbar_arrive(&bars[kOutFree]);
                    }
#pragma unroll
                    for (int jj = 0; jj < 32; jj += 2) {
                        float s0 = p.scale, s1 = p.scale;
                        if constexpr (!BF) {
                            const float2 two = *reinterpret_cast<const float2 *>(row_scale + 128 + 32 * b + jj);
                            s0 = two.x;
                            s1 = two.y;
                        }
                        const uint32_t two = pack2<BF>(fmaf(__uint_as_float(r[jj]), s0, hold[32 * b + jj]),
                                                       fmaf(__uint_as_float(r[jj + 1]), s1, hold[32 * b + jj + 1]));
                        stage[(32 * b + jj) * 128] = static_cast<unsigned short>(two);
                        stage[(32 * b + jj + 1) * 128] = static_cast<unsigned short>(two >> 16);
                    }
                }
                if (!(ok = group_sync(&bars[kSyncA], ph))) break;
                const int piece = tid & 15, tok = tid >> 4;
                unsigned short *o = out + (un.t0 + c + tok) * p.os[0] + 8 * piece;
                const unsigned char *from = smem + LY::kP + tid * 16;
                const int64_t step = 8 * p.os[0];
                if (8 * piece < p.P) {
#pragma unroll 4
                    for (int i = 0; i < 16; ++i)
                        if (tok + 8 * i < n)
                            *reinterpret_cast<uint4 *>(o + i * step) = *reinterpret_cast<const uint4 *>(from + i * 2048);
                }
                // P's place, and the score rows' scales, are read
                if (!(ok = group_sync(&bars[kSyncA], ph))) break;
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) flag(p.status, kDevTimeout);
            *abort_flag = 1;
        }
    } else {
        registers<216>();
        // ---------------- the state and the decayed values ----------------
        const int t = tid - kGroup, w = warp - 4;  // value dim
        const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
        float *tab = reinterpret_cast<float *>(smem + LY::kTabB);
        float *row_scale = reinterpret_cast<float *>(smem + LY::kRowScale);
        float *maxes = reinterpret_cast<float *>(smem + LY::kMax);
        int nu = 0, ch = 0, quarters = 0, ph = 0;
        float S[DK];
        for (;;) {
            if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
            const Unit un = ring[nu & 1];
            mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
            ++nu;
            if (un.len < 0) break;
            const float g = fmaxf(__ldg(p.log_decay + un.h), -1e30f);
            if (!(ok = group_sync(&bars[kSyncB], ph))) break;  // the previous unit's table is no longer read
            tab[t] = expf(g * static_cast<float>(kC - 1 - t));
            if (t < kQuarter) tab[kC + t] = 0.f;
            const float lam_chunk = expf(g * static_cast<float>(kC));
            // the entering state: this thread's row
#pragma unroll
            for (int i = 0; i < DK; ++i) S[i] = 0.f;
            if (un.src != kZero && t < p.P) {
                const int64_t at = ((un.src * p.H + un.h) * static_cast<int64_t>(p.P) + t) * p.N;
                if (p.state_dtype == kF32) {
#pragma unroll
                    for (int i = 0; i < DK; i += 4)
                        if (i < p.N) StateChunk<float>::unpack(ld_stream(static_cast<const float *>(p.state) + at + i), S + i);
                } else if (p.state_dtype == kBF16) {
#pragma unroll
                    for (int i = 0; i < DK; i += 8)
                        if (i < p.N)
                            StateChunk<__nv_bfloat16>::unpack(ld_stream(static_cast<const __nv_bfloat16 *>(p.state) + at + i), S + i);
                } else {
#pragma unroll
                    for (int i = 0; i < DK; i += 8)
                        if (i < p.N) StateChunk<__half>::unpack(ld_stream(static_cast<const __half *>(p.state) + at + i), S + i);
                }
            }
            if (!(ok = group_sync(&bars[kSyncB], ph))) break;
            for (int c = 0; c < un.len; c += kC, ++ch) {
                const int s = ch & 1, n = min(kC, un.len - c);
                // S in two parts, for the entering product (where the last
                // chunk's decayed V was, which its growth product has read)
                float sc = 1.f;
                if constexpr (!BF) {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < DK; ++i) m = fmaxf(m, fabsf(S[i]));
                    const int k = fp16_scale_exp(m);
                    sc = pow2i(k);
                    // read before kPFull, which the growth product that this
                    // thread waits for below comes after
                    row_scale[t] = pow2i(-k);
                }
#pragma unroll
                for (int b = 0; b < DK / 32; ++b) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = S[32 * b + 2 * i] * sc, y = S[32 * b + 2 * i + 1] * sc;
                        hi[i] = pack2<BF>(x, y);
                        const float2 f = unpack2<BF>(hi[i]);
                        lo[i] = pack2<BF>(x - f.x, y - f.y);
                    }
                    tmem_st16(tmem + lanes + kColState + 16 * b, hi);
                    tmem_st16(tmem + lanes + kColState + DK / 2 + 16 * b, lo);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars[kStateFull]);
                if (!(ok = mbar_wait_bounded(&bars[kFull0 + s], (ch >> 1) & 1))) break;
                unsigned char *sK = smem + s * LY::kStage + LY::kQBytes, *sV = sK + LY::kKBytes;
                if (n < kC) {
                    // rows past the piece's end belong to other tokens: a
                    // weight of zero would still let their NaN through
                    constexpr int kPanels = DK / 64 + 2;
                    for (int i = t; i < (kC - n) * 8 * kPanels; i += kGroup) {
                        const int at = i % ((kC - n) * 8);
                        *reinterpret_cast<uint4 *>(sK + (i / ((kC - n) * 8)) * kPanel + n * 128 + at * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[kTail]);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;  // every thread's zeros, below
                }
                float vs = 1.f, vback = 1.f;
                if constexpr (!BF) {
                    // the power of two that brings the tile's largest |v| near fp16's top
                    uint32_t m2 = 0u;
                    for (int i = t; i < 2 * kPanel / 16; i += kGroup) {
                        if ((i % (kPanel / 16)) / 8 >= n) continue;
                        const uint4 u = *reinterpret_cast<const uint4 *>(sV + i * 16);
                        const uint32_t ws[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint32_t a = ws[e] & 0x7fff7fffu;
                            m2 = __vmaxu2(m2, a);  // magnitudes order as their bits
                        }
                    }
                    float m = fmaxf(__half2float(__ushort_as_half(static_cast<unsigned short>(m2))),
                                    __half2float(__ushort_as_half(static_cast<unsigned short>(m2 >> 16))));
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                    if (lane == 0) maxes[w] = m;
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    m = fmaxf(fmaxf(maxes[0], maxes[1]), fmaxf(maxes[2], maxes[3]));
                    const int k = fp16_scale_exp(m);
                    vs = pow2i(k);
                    vback = pow2i(-k);
                }
                // the decayed V, 32 tokens at a time, where the parts of S were
                if (!(ok = mbar_wait_bounded(&bars[kEnter], ch & 1))) break;
                tc_fence_after();
                // (column t of V: the swizzle moves its 16-byte piece with the row)
                const unsigned char *vcol = sV + (t >> 6) * kPanel + (t & 7) * 2;
                const int piece = ((t & 63) >> 3) * 16;
                const float *weight = tab + (kC - n);
                for (int q0 = 0; q0 < n; q0 += kQuarter, ++quarters) {
                    const int r = quarters & 1;
                    float x[kQuarter];
#pragma unroll
                    for (int j = 0; j < kQuarter; j += 4) {
                        float we[4];
                        if (n == kC) {
                            const float4 wj = *reinterpret_cast<const float4 *>(weight + q0 + j);
                            we[0] = wj.x, we[1] = wj.y, we[2] = wj.z, we[3] = wj.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) we[e] = weight[q0 + j + e];
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const unsigned short u = *reinterpret_cast<const unsigned short *>(
                                vcol + q0 * 128 + (j + e) * 128 + (piece ^ (((j + e) & 7) * 16)));
                            const float v =
                                BF ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u)) * vs;
                            x[j + e] = v * we[e];
                        }
                    }
                    if (quarters >= 2 && !(ok = mbar_wait_bounded(&bars[kVFree0 + r], ((quarters >> 1) - 1) & 1))) break;
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < kParts; ++q) {
                        uint32_t part[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if constexpr (BF) {
                                // the top 8 bits of what is left: three parts hold all 24
                                const uint32_t a = __float_as_uint(x[2 * i]), c2 = __float_as_uint(x[2 * i + 1]);
                                part[i] = __byte_perm(a, c2, 0x7632);
                                x[2 * i] -= __uint_as_float(a & 0xffff0000u);
                                x[2 * i + 1] -= __uint_as_float(c2 & 0xffff0000u);
                            } else {
                                part[i] = pack2<BF>(x[2 * i], x[2 * i + 1]);
                                const float2 f = unpack2<BF>(part[i]);
                                x[2 * i] -= f.x;
                                x[2 * i + 1] -= f.y;
                            }
                        }
                        tmem_st16(tmem + lanes + kColState + r * kRing + 16 * q, part);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(&bars[kVFull0 + r]);
                }
                if (!ok) break;
                mbar_arrive(&bars[kFree0 + s]);
                if (!(ok = mbar_wait_bounded(&bars[kGrowth], ch & 1))) break;
                tc_fence_after();
                const float lam = n == kC ? lam_chunk : expf(g * static_cast<float>(n));
#pragma unroll
                for (int b = 0; b < DK / 32; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kColGrowth + 32 * b, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[32 * b + i] = fmaf(S[32 * b + i], lam, __uint_as_float(r[i]) * vback);
                }
                tc_fence_before();
            }
            if (!ok) break;
            if (un.dst != kNone && t < p.P) {
                const int64_t at = ((un.dst * p.H + un.h) * static_cast<int64_t>(p.P) + t) * p.N;
                if (p.state_dtype == kF32) {
#pragma unroll
                    for (int i = 0; i < DK; i += 4)
                        if (i < p.N) st_stream(static_cast<float *>(p.state) + at + i, StateChunk<float>::pack(S + i));
                } else if (p.state_dtype == kBF16) {
#pragma unroll
                    for (int i = 0; i < DK; i += 8)
                        if (i < p.N) st_stream(static_cast<__nv_bfloat16 *>(p.state) + at + i, StateChunk<__nv_bfloat16>::pack(S + i));
                } else {
#pragma unroll
                    for (int i = 0; i < DK; i += 8)
                        if (i < p.N) st_stream(static_cast<__half *>(p.state) + at + i, StateChunk<__half>::pack(S + i));
                }
            }
        }
        if (!ok) {
            if (lane == 0) flag(p.status, kDevTimeout);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc512(tmem);
}

// The driver's tensor-map encoder, looked up once.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                              const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// [rows, heads, n] 16-bit elements: boxes of 128 rows of one head by 64
// elements, zeros past n and past the last row.
bool encode(CUtensorMap *m, const LinattnParams &p, const void *base, int n, int heads, const int64_t *stride) {
    const EncodeFn fn = encoder();
    if (!fn) return false;
    // a stride along an extent of one is never used; keep it legal
    const int64_t hs = heads > 1 ? stride[1] : n, ts = p.rows > 1 ? stride[0] : static_cast<int64_t>(n) * heads;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(p.rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2, static_cast<cuuint64_t>(ts) * 2};
    const cuuint32_t box[3] = {64, 1, kC}, unit[3] = {1, 1, 1};
    const CUtensorMapDataType type = p.io_dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, type, 3, const_cast<void *>(base), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static int cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 0 || dev >= 64) dev = 0;
    int n = __atomic_load_n(&cache[dev], __ATOMIC_RELAXED);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        __atomic_store_n(&cache[dev], n, __ATOMIC_RELAXED);
    }
    return n;
}

template <int DK, bool BF>
cudaError_t launch_t(const LinattnParams &p, cudaStream_t stream) {
    Maps maps;
    if (p.rows > 0 && !(encode(&maps.q, p, p.q, p.N, p.H, p.qs) && encode(&maps.k, p, p.k, p.N, p.G, p.ks) &&
                        encode(&maps.v, p, p.v, p.P, p.G, p.vs)))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(linattn_prefill_kernel<DK, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Layout<DK>::kBytes);
    if (e != cudaSuccess) return e;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    const int64_t units = p.nseq * p.H;
    const int64_t grid = units < sms ? units : sms;
    linattn_prefill_kernel<DK, BF><<<static_cast<unsigned>(grid), kThreads, Layout<DK>::kBytes, stream>>>(p, maps, units);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_prefill(const LinattnParams &p, cudaStream_t stream) {
    const bool bf = p.io_dtype == kBF16;
    if (p.N <= 64) return bf ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
    return bf ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
}

}  // namespace ssu
