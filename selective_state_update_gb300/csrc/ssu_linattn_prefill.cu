// ssu_linattn_prefill.cu -- linear attention with a decay for each head over
// packed prompts: the chunked form on the 5th-generation tensor cores.
//
// The recurrence S_t = l S_{t-1} + v_t k_t^T, out_t = scale S_t q_t, l =
// e^log_decay[h], over a chunk of n <= 128 tokens (i, j within it) with S the
// state that enters it:
//     out_i = scale (l^(i+1) S q_i + sum_{j<=i} l^(i-j) (q_i . k_j) v_j)
//     S'    = l^n S + sum_j l^(n-1-j) v_j k_j^T
// A work unit is one piece of a sequence -- the whole of it, or an equal part of
// a long one -- for one head; a CTA walks its chunks and carries S in registers.
//
// Calls with more (sequence, head) pairs than SMs are planned by a small kernel
// first: it checks the metadata, cuts sequences longer than a given length into
// pieces and orders the pieces by length, longest first, from where the CTAs
// take them in turn.  Where sequences are cut, two more kernels run before the
// main one: this one again for what each piece adds to the state (the growth
// products alone), and a pass along each cut sequence that turns those into
// the states that enter its pieces.
//
// Four products a chunk, tcgen05.mma with fp32 accumulators in tensor memory:
//   scores   [i, j]  = Q K^T            Q, K from shared memory, as loaded
//   entering [i, p]  = Q S^T            S rounded to the io type, in shared memory
//   inside   [i, p] += P V              P = scores decayed and masked, rounded once, from
//                                       tensor memory; added to the entering product,
//                                       whose rows have been scaled there by l^(i+1) in fp32
//   growth   [p, n]  = (V decayed)^T K  the decayed V in three parts (bf16) or two
//                                       (fp16), transposed, from tensor memory
// Rounding: P and, where it meets Q, S to the io type (2^-8 bf16, 2^-11 fp16),
// each once; the decayed V to three parts (2^-24) or two (2^-22), so that fp32
// states keep fp32 accuracy.  The first two cost the outputs u sum |P| |V| and
// u |S| |Q|, u being the io type's rounding: as much as one more rounding of Q
// or V, which the caller has rounded to the same type.  On normal inputs in
// bf16 the outputs are off by 0.0023 of their norm, where their own rounding
// alone is 0.0017 of it; where a sum cancels it is more beside the output.  S in
// two parts as well took 260 us where one took 235 (32768 tokens x 32 heads):
// eight more products, and the shared memory that the second Q now has.  fp16
// operands are scaled by powers of two (per state row, score row and chunk of
// values), so neither overflow nor the subnormals cost accuracy.
//
// Warps, in groups of four (a warp reaches the tensor-memory lanes 32 (warp %
// 4) ...):
//   0-3    (thread = token) scores -> P, entering rows scaled, outputs stored;
//   4-7    (thread = value dim) S: growth added, parts split off, first and last state;
//   8-11   V decayed, transposed (ldmatrix) and split, 32 tokens at a time, and
//          looked through for what is no number;
//   12     issues the products;  13 finds the units and loads Q, K, V by tiled copies,
//          two chunks ahead of the outputs, which leave through Q's place;
//   14     stores the outputs by tiled copies;  15 only completes the group.
// The groups' code for a chunk is kept short (loops over blocks and quarters are
// not unrolled): all of it together has to stay in the instruction cache
// (unrolled, 384 us instead of 257 at that stage).
//
// What it takes: 32768 tokens in 16 sequences x 32 heads of 128 x 128 (bf16, fp32
// states, some read) 229 us, 4.9 TB/s of the bytes that have to move, 0.72 of the
// copy rate; one sequence of 40001 tokens x 16 heads (4 of keys) 186 us, of which the
// growth pass 60.  A chunk takes 2.95 us on every SM at once (3.3 with keys and
// values of its own for every head, 3.8 in fp16): 48 products of 128 x 128 x 16 and
// more keep the tensor pipe at work for 3.1 thousand cycles of it, the others go
// to the hand-overs between the groups; its 450 KB of shared-memory traffic would
// take 3.5 thousand.  A unit of one token takes 12 us by itself, launch and cold
// instructions included.
#include <cuda.h>

#include "ssu_hybrid.h"
#include "ssu_tcgen05.cuh"

namespace ssu {

namespace {

constexpr int kC = 128;        // tokens of a chunk
constexpr int kPanel = 16384;  // 128 rows of 128 bytes
constexpr int kThreads = 512;
constexpr int kGroup = 128;    // threads of a group of four warps
constexpr int kQuarter = 32;   // tokens whose decayed V is handed over at a time

// Tensor-memory columns.  P goes where its scores were.
constexpr uint32_t kColScore = 0, kColOut = 128, kColGrowth = 256, kColV = 384;
constexpr uint32_t kRing = 48;  // columns of one quarter: up to 3 parts of 16

struct Unit {
    int64_t t0;   // first token row
    int64_t src;  // state entering: pool slot, kZero, or kScratch + state of the workspace
    int64_t dst;  // state leaving: pool slot or kNone
    int32_t len;  // tokens; -1: no more units
    int32_t h;    // head; in the plan: not the last piece of its sequence
};
constexpr int64_t kZero = -1, kNone = -1, kScratch = int64_t(1) << 62;

// The plan in the workspace: counters, the cut sequences, the pieces.
struct Cut {
    int32_t state, pieces;  // first workspace state, number of pieces
    int64_t src, len;       // the sequence's first state and length
};
struct PlanHead {
    int32_t pieces, cuts;
    int32_t next[2];  // the next unit of the growth pass and of the main one
};
struct Plan {
    PlanHead *head;  // nullptr: a unit is (sequence, head), found on the spot
    Cut *cuts;
    Unit *pieces;
    float *states;   // [state][head][dim][dstate]
    int64_t cut_len;  // longest piece, a multiple of kC
    int64_t max_cuts, max_states;  // what the workspace has room for
};

enum : int {
    kQFull0, kQFull1,  // a Q has landed
    kQFree0, kQFree1,  // ... and is done with, and the outputs in its place are stored
    kFull0, kFull1,    // a stage's K and V have landed
    kFree0, kFree1,    // ... and are done with
    kUnitFull0, kUnitFull1, kUnitFree0, kUnitFree1,
    kScore,            // the scores are there
    kStateFull,        // the rounded S is there
    kEnter,            // the entering product is there (S and Q are read)
    kPFull,            // P is there, the entering product scaled
    kInside,           // the outputs are there (P is read)
    kOutFree,          // ... and read
    kStaged0, kStaged1,  // ... and laid out by token, in Q's place; one for each stage, as the outputs of the next
                       // chunk may come before the store of this one's has been begun
    kTail0, kTail1,    // a stage's partial chunk has zeros past its end; one for each stage, whose kFree keeps
                       // the next such chunk from completing it before this one has been waited for
    kVFull0, kVFull1, kVFree0, kVFree1,
    kGrowth, kGrowthFree,
    kSyncA, kSyncB, kSyncC,
    kFinal,
    kGrowth1, kGrowthFree1,  // the growth pass's second growth
    kBars
};

template <int DK>
struct Layout {
    static constexpr int kPanels = DK / 64;
    static constexpr int kKBytes = kPanels * kPanel;
    static constexpr int kVBytes = 2 * kPanel;
    static constexpr int kStage = kKBytes + kVBytes;
    static constexpr int kQ = 2 * kStage;                 // two, each with room for two panels of outputs
    static constexpr int kQBytes = 2 * kPanel;
    static constexpr int kS = kQ + 2 * kQBytes;           // kPanels panels
    static constexpr int kBar = kS + kKBytes;
    static constexpr int kUnits = kBar + 8 * kBars;       // Unit[2]
    static constexpr int kRowScale = (kUnits + 2 * static_cast<int>(sizeof(Unit)) + 15) / 16 * 16;  // fp16: state rows, by chunk parity
    static constexpr int kMax = kRowScale + 2 * 128 * 4;  // fp16: per warp; the value tiles' scales, four chunks; per warp of the growth pass's helpers
    static constexpr int kMisc = kMax + 48;               // tensor-memory address, abort
    static constexpr int kOdd = kMisc + 16;               // by chunk, of four, and warp of value dims: the last chunk with
    static constexpr int kFirst = kOdd + 4 * 16;          // values that are no numbers; of every dim the token of its first
    static constexpr int kBytes = kFirst + 4 * 128;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

struct Maps {
    CUtensorMap q, k, v, out;
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
// Two floats as parts of the io type, the largest first; x, y are left with
// the rest.  bf16: the top 16 bits, so that three parts hold all 24 bits of a
// float's mantissa.
template <bool BF>
__device__ __forceinline__ uint32_t split2(float &x, float &y) {
    if constexpr (BF) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        x -= __uint_as_float(a & 0xffff0000u);
        y -= __uint_as_float(b & 0xffff0000u);
        return __byte_perm(a, b, 0x7632);
    } else {
        const uint32_t u = pack2<BF>(x, y);
        const float2 f = unpack2<BF>(u);
        x -= f.x;
        y -= f.y;
        return u;
    }
}

// Gives up (N below the launch's 128) or takes registers; every warp of a group
// of four calls it with the same N.
template <int N>
__device__ __forceinline__ void registers() {
    if constexpr (N < 128) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
    else if constexpr (N > 128) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Four 8 x 8 matrices of 16-bit elements, transposed: the lane's address is row
// lane % 8 of matrix lane / 8; register m gets, of matrix m, rows 2 (lane % 4)
// and + 1 of column lane / 4.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t saddr, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
// 16 lanes x 16 columns: register 2 c + i goes to lane 8 i + lane / 4, column
// 4 c + lane % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    tmem_st16(taddr, r);
    tmem_st16(taddr + 16, r + 16);
}

// Where element `dim` of row `row` lies in panels of 64 16-bit elements a row.
__device__ __forceinline__ int swizzled(int row, int dim) {
    return (dim >> 6) * kPanel + row * 128 + ((((dim & 63) >> 3) ^ (row & 7)) * 16) + (dim & 7) * 2;
}
// sum += 0 v, two bf16 each: a NaN from the first v on that is no number.
__device__ __forceinline__ void add_zero_times(uint32_t &sum, uint32_t v) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(v), "r"(0u));
}
// A NaN or an infinity among a chunk's values would reach the outputs of the
// tokens before it, by a zero of P.  So they are made zeros in shared memory, where
// P meets them, once they have been read for the state; and the rows' group
// makes the outputs of a dim NaN from the first one's token on, which this returns
// (kC where there is none).  Looking for them, and the room that this takes in the
// instruction cache, costs 2 to 4 % (232 us for 223, 32768 tokens x 32 heads).  A
// warp of its own that looked through every chunk cost 14 %, the products' warp
// asking for it 5.
template <bool BF>
__device__ __forceinline__ int take_out(unsigned char *values, int dim, int tokens) {
    int first = kC;
#pragma unroll 1
    for (int row = tokens - 1; row >= 0; --row) {
        unsigned short *v = reinterpret_cast<unsigned short *>(values + swizzled(row, dim));
        if ((*v & 0x7fff) < (BF ? 0x7f80 : 0x7c00)) continue;
        *v = 0;
        first = row;
    }
    fence_proxy_async_smem();
    return first;
}

// A head's state [P][N] between memory (T, contiguous) and the state's place in
// shared memory, 16 bytes a thread along memory, for one group of warps.  The
// place holds kCols columns of every row at a time; its 16-byte pieces are swapped
// by row, so that the threads' own rows are read and written without bank
// conflicts.
template <typename T, int DK>
struct StateRow {
    static constexpr int kVec = 16 / static_cast<int>(sizeof(T));
    static constexpr int kCols = 2 * DK / static_cast<int>(sizeof(T));  // the place has 2 DK bytes a row
    __device__ __forceinline__ static int at(int row, int piece) { return row * 2 * DK + ((piece ^ (row & 7)) * 16); }
};
template <typename T, int DK, typename F>
__device__ __forceinline__ void each_piece(int P, int N, int c0, int t, F f) {
    using R = StateRow<T, DK>;
    const int per = min(R::kCols, N - c0) / R::kVec, total = P * per, down = kGroup / per, right = kGroup - down * per;
    int row = t / per, piece = t - row * per;
#pragma unroll 4
    for (int i = t; i < total; i += kGroup) {
        f(row * N + c0 + piece * R::kVec, R::at(row, piece));
        row += down;
        piece += right;
        if (piece >= per) piece -= per, ++row;
    }
}
template <typename T, int DK>
__device__ __forceinline__ void stage_in(const T *src, unsigned char *place, int P, int N, int c0, int t) {
    each_piece<T, DK>(P, N, c0, t, [&](int i, int at) { cp16(place + at, src + i, true); });
    cp_wait_all();
}
template <typename T, int DK>
__device__ __forceinline__ void stage_out(T *dst, const unsigned char *place, int P, int N, int c0, int t) {
    each_piece<T, DK>(P, N, c0, t, [&](int i, int at) { st_stream(dst + i, *reinterpret_cast<const uint4 *>(place + at)); });
}
// Columns C0 ... of this thread's row.
template <typename T, int DK, int C0>
__device__ __forceinline__ void row_from(const unsigned char *place, int row, int N, float *S) {
    using R = StateRow<T, DK>;
#pragma unroll
    for (int j = 0; j < R::kCols / R::kVec; ++j)
        if (C0 + j * R::kVec < N)
            StateChunk<T>::unpack(*reinterpret_cast<const uint4 *>(place + R::at(row, j)), S + C0 + j * R::kVec);
}
template <typename T, int DK, int C0>
__device__ __forceinline__ void row_to(unsigned char *place, int row, const float *S) {
    using R = StateRow<T, DK>;
#pragma unroll
    for (int j = 0; j < R::kCols / R::kVec; ++j)
        *reinterpret_cast<uint4 *>(place + R::at(row, j)) = StateChunk<T>::pack(S + C0 + j * R::kVec);
}

// `bytes` (a multiple of 16, 16-byte aligned) into L2.
__device__ __forceinline__ void bulk_prefetch(const void *p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Sequence b: its bounds and slots.  False (and flagged) when it is to be
// skipped.
__device__ __forceinline__ bool find_sequence(const LinattnParams &p, int64_t b, Unit &out) {
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

// How a sequence of `len` tokens is cut: pieces of `step` tokens, the last one
// shorter.
__device__ __forceinline__ int piece_count(int64_t len, int64_t cut_len) {
    return len <= cut_len ? 1 : static_cast<int>((len + cut_len - 1) / cut_len);
}
__device__ __forceinline__ int64_t piece_step(int64_t len, int pieces) {
    return ((len + pieces - 1) / pieces + kC - 1) / kC * kC;
}

// One CTA: pieces counted into buckets by their chunks, then placed, longest
// first (the order within a bucket is free: it decides who works when, not on
// what).
constexpr int kPlanThreads = 1024, kBuckets = 1024;
__global__ void __launch_bounds__(kPlanThreads) linattn_plan_kernel(const LinattnParams p, const Plan plan, int grid) {
    __shared__ int start[kBuckets];
    __shared__ int warp_sum[32];
    __shared__ int states, cuts;
    __shared__ unsigned long long want_states, want_cuts;
    const int tid = threadIdx.x;
    start[tid] = 0;
    if (tid == 0) states = cuts = 0, want_states = want_cuts = 0;
    __syncthreads();
    Unit own;  // this thread's first sequence is looked up once
    bool have = false;
    for (int64_t b = tid; b < p.nseq; b += kPlanThreads) {
        Unit un;
        const bool ok = find_sequence(p, b, un);
        if (b == tid) own = un, have = ok;
        const int n = ok ? piece_count(un.len, plan.cut_len) : 1;
        if (n > 1) {
            atomicAdd(&want_cuts, 1ull);
            atomicAdd(&want_states, static_cast<unsigned long long>(n));
        }
    }
    __syncthreads();
    // Sequences that follow one another fit the workspace.  Bounds that go back
    // and forth may name more tokens than there are: then none is cut.
    const int64_t cut_len =
        want_cuts <= static_cast<unsigned long long>(plan.max_cuts) && want_states <= static_cast<unsigned long long>(plan.max_states)
            ? plan.cut_len
            : int64_t(1) << 40;
    LinattnParams quiet = p;
    quiet.status = nullptr;  // flagged above
    const auto sequence = [&](int64_t b, Unit &un) {
        if (b != tid) return find_sequence(quiet, b, un);
        un = own;
        return have;
    };
    const auto bucket = [](int64_t len) { return kBuckets - 1 - static_cast<int>(min((len + kC - 1) / kC, int64_t(kBuckets - 1))); };
    // step s of a cut sequence may leave fewer pieces than counted: n pieces of
    // `step` tokens, the last of what is left
    const auto each = [&](const Unit &un, auto f) {
        const int n0 = piece_count(un.len, cut_len);
        const int64_t step = n0 == 1 ? un.len : piece_step(un.len, n0);
        const int n = n0 == 1 ? 1 : static_cast<int>((un.len + step - 1) / step);
        for (int i = 0; i < n; ++i) f(i, n, min(step, un.len - i * step), i * step);
    };
    for (int64_t b = tid; b < p.nseq; b += kPlanThreads) {
        Unit un;
        if (sequence(b, un)) each(un, [&](int, int, int64_t len, int64_t) { atomicAdd(&start[bucket(len)], 1); });
    }
    __syncthreads();
    // exclusive prefix sum of the buckets
    const int lane = tid & 31, warp = tid >> 5, mine = start[tid];
    int sum = mine;
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += o;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    start[tid] = before + sum - mine;
    __syncthreads();
    for (int64_t b = tid; b < p.nseq; b += kPlanThreads) {
        Unit un;
        if (!sequence(b, un)) continue;
        int state = 0, cut = 0;
        each(un, [&](int i, int n, int64_t len, int64_t off) {
            if (i == 0 && n > 1) {
                state = atomicAdd(&states, n);
                cut = atomicAdd(&cuts, 1);
                plan.cuts[cut] = Cut{state, n, un.src, un.len};
            }
            Unit piece;
            piece.t0 = un.t0 + off;
            piece.len = static_cast<int>(len);
            piece.src = n > 1 ? kScratch + state + i : un.src;
            piece.dst = i == n - 1 ? un.dst : kNone;
            piece.h = i < n - 1;
            plan.pieces[atomicAdd(&start[bucket(len)], 1)] = piece;
        });
    }
    __syncthreads();
    if (tid == 0) *plan.head = PlanHead{total, cuts, {grid, grid}};
}

// Along each cut sequence: what its pieces add becomes what enters them.
__global__ void __launch_bounds__(256) linattn_carry_kernel(const LinattnParams p, const Plan plan) {
    if (static_cast<int>(blockIdx.z) >= plan.head->cuts) return;
    const Cut cut = plan.cuts[blockIdx.z];
    const int h = blockIdx.y;
    const int64_t elems = static_cast<int64_t>(p.P) * p.N, at = (blockIdx.x * 256 + threadIdx.x) * int64_t(4);
    if (at >= elems) return;
    const float g = fmaxf(__ldg(p.log_decay + h), -1e30f);
    const int64_t step = piece_step(cut.len, piece_count(cut.len, plan.cut_len));
    const float lam = expf(g * static_cast<float>(step));
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (cut.src != kZero) {
        const int64_t i = (cut.src * p.H + h) * elems + at;
        for (int e = 0; e < 4; ++e)
            s[e] = p.state_dtype == kF32 ? static_cast<const float *>(p.state)[i + e]
                                         : bits_to_float(static_cast<const unsigned short *>(p.state)[i + e], p.state_dtype);
    }
    float4 *w = reinterpret_cast<float4 *>(plan.states + (static_cast<int64_t>(cut.state) * p.H + h) * elems + at);
    const int64_t stride = p.H * elems / 4;
    constexpr int kBatch = 8;  // loads in flight; the sums along the pieces depend on one another
    for (int i0 = 0; i0 < cut.pieces; i0 += kBatch, w += kBatch * stride) {
        float4 add[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            add[i] = i0 + i < cut.pieces - 1 ? w[i * stride] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (i0 + i >= cut.pieces) break;
            w[i * stride] = make_float4(s[0], s[1], s[2], s[3]);
            s[0] = fmaf(s[0], lam, add[i].x);
            s[1] = fmaf(s[1], lam, add[i].y);
            s[2] = fmaf(s[2], lam, add[i].z);
            s[3] = fmaf(s[3], lam, add[i].w);
        }
    }
}

// GROW: only what the pieces add to the state, into the workspace.
template <int DK, bool BF, bool GROW>
__global__ void __launch_bounds__(kThreads, 1)
    linattn_prefill_kernel(const LinattnParams p, const __grid_constant__ Maps maps, const Plan plan) {
    using LY = Layout<DK>;
    constexpr int kParts = BF ? 3 : 2;  // parts of the decayed V
    // The growth pass has the outputs' columns free and lets the chunks' growths
    // take turns there, so that one is read while the next is formed.
    const auto growth_at = [](int ch) { return GROW && (ch & 1) ? kColOut : kColGrowth; };
    const auto growth_bar = [](int ch) { return GROW && (ch & 1) ? kGrowth1 : kGrowth; };
    const auto growth_free = [](int ch) { return GROW && (ch & 1) ? kGrowthFree1 : kGrowthFree; };
    const auto growth_phase = [](int ch) { return GROW ? ch >> 1 : ch; };
    extern __shared__ __align__(1024) unsigned char smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + LY::kBar);
    Unit *ring = reinterpret_cast<Unit *>(smem + LY::kUnits);
    uint32_t *misc = reinterpret_cast<uint32_t *>(smem + LY::kMisc);
    float *row_scale = reinterpret_cast<float *>(smem + LY::kRowScale);
    float *maxes = reinterpret_cast<float *>(smem + LY::kMax);
    volatile uint32_t *abort_flag = misc + 1;
    int *odd_chunk = reinterpret_cast<int *>(smem + LY::kOdd);
    unsigned char *first_odd = smem + LY::kFirst;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kBars; ++i) {
            int n = 1;
            if (i == kFree0 || i == kFree1) n = 1 + (GROW ? 2 : 1) * kGroup;
            if (i == kUnitFree0 || i == kUnitFree1) n = (GROW ? 1 : 2) + 3 * kGroup;
            if (i == kStateFull || i == kPFull || i == kOutFree || i == kStaged0 || i == kStaged1 || i == kTail0 || i == kTail1 ||
                i == kVFull0 || i == kVFull1 || i == kGrowthFree || i == kGrowthFree1 || i == kSyncA || i == kSyncB || i == kSyncC)
                n = kGroup;
            mbar_init(&bars[i], n);
        }
        for (int i = 0; i < 16; ++i) odd_chunk[i] = -1;
        *abort_flag = 0;
    }
    if (warp == 12) tmem_alloc512(misc);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    bool ok = true;

    // The decayed values (warp = 32 value dims), by the third group of warps; in
    // the growth pass the first one, `helper` 1, takes every second quarter.
    const auto decay_values = [&](int helper) {
        const int sync = helper ? kSyncA : kSyncC;
        uint32_t *tile_max = reinterpret_cast<uint32_t *>(maxes + (helper ? 8 : 0));
        const int t = tid % kGroup, w = warp % 4;
        const bool live = 32 * w < p.P;
        int nu = 0, ch = 0, quarters = 0, ph = 0;
        // this lane's row of the matrices it loads: token lane % 8 of token
        // block lane / 16 of two, 8 value dims of block (lane / 8) % 2; the
        // swizzle moves the 16-byte piece with the token
        const int dim0 = 32 * w + 8 * ((lane >> 3) & 1);
        uint32_t at[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int d = dim0 + 16 * hh;
            at[hh] = smem_addr(smem) + LY::kKBytes + (d >> 6) * kPanel + ((lane & 7) + 8 * (lane >> 4)) * 128 +
                     ((((d & 63) >> 3) ^ (lane & 7)) * 16);
        }
        for (;;) {
            if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
            const Unit un = ring[nu & 1];
            mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
            ++nu;
            if (un.len < 0) break;
            const float g = fmaxf(__ldg(p.log_decay + un.h), -1e30f);
            float fall[8];  // l^(31 - j) of this lane's tokens j = 8 b + 2 (lane % 4) + e of a quarter
#pragma unroll
            for (int i = 0; i < 8; ++i) fall[i] = expf(g * static_cast<float>(31 - 8 * (i >> 1) - 2 * (lane & 3) - (i & 1)));
            for (int c = 0; c < un.len; c += kC, ++ch) {
                const int s = ch & 1, n = min(kC, un.len - c);
                if (!(ok = mbar_wait_bounded(&bars[kFull0 + s], (ch >> 1) & 1))) break;
                unsigned char *sK = smem + s * LY::kStage;
                if (n < kC) {
                    // rows past the sequence's end belong to other tokens: a
                    // weight of zero would still let their NaN through
                    // (as far as a product or the decay below reads them)
                    const int pieces = ((n + kQuarter - 1) / kQuarter * kQuarter - n) * 8;
                    for (int panel = 0; panel < LY::kPanels + (p.P > 64 ? 2 : 1); ++panel)
                        for (int i = t; i < pieces; i += kGroup)
                            *reinterpret_cast<uint4 *>(sK + panel * kPanel + n * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[kTail0 + s]);
                    if (!(ok = group_sync(&bars[sync], ph))) break;  // every thread's zeros, below
                }
                float vs = 1.f;
                bool odd = false;  // some of the warp's values (fp16: of the chunk's) are no numbers
                if constexpr (!BF) {
                    // the power of two that brings the chunk's largest |v| near
                    // fp16's top (the rows past its end are zeros as far as the
                    // last quarter goes, and after it other tokens')
                    uint32_t pair = 0u;
                    const int turns = (n + kQuarter - 1) / kQuarter * 2;  // a turn takes 16 rows of 8 pieces
                    const auto largest = [](uint4 u) {                    // magnitudes order as their bits
                        return __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
                    };
                    for (int panel = 0; panel < (p.P > 64 ? 2 : 1); ++panel) {
                        const unsigned char *from = sK + LY::kKBytes + panel * kPanel + t * 16;
#pragma unroll 1
                        for (int i = 0; i < turns; i += 2, from += 2 * kGroup * 16)
                            pair = __vmaxu2(pair, __vmaxu2(largest(*reinterpret_cast<const uint4 *>(from)),
                                                           largest(*reinterpret_cast<const uint4 *>(from + kGroup * 16))));
                    }
                    uint32_t m = max(pair & 0xffffu, pair >> 16);
                    if (__builtin_expect(m >= 0x7c00u, 0)) {  // no number: the largest of the others, and a mark
                        m = 0u;
#pragma unroll 1
                        for (int i = t * 8; i < (p.P > 64 ? 2 : 1) * (kPanel / 2); i += (i & 7) == 7 ? kGroup * 8 - 7 : 1) {
                            const uint32_t x = reinterpret_cast<const unsigned short *>(sK + LY::kKBytes)[i] & 0x7fffu;
                            if ((i / 64 & (kC - 1)) < n && x < 0x7c00u) m = max(m, x);
                        }
                        m |= 0x10000u;
                    }
                    odd = __any_sync(0xffffffffu, m > 0xffffu);
                    m = __reduce_max_sync(0xffffffffu, m & 0xffffu);
                    if (lane == 0) tile_max[w] = odd ? m | 0x10000u : m;
                    if (!(ok = group_sync(&bars[sync], ph))) break;
                    const uint32_t m0 = tile_max[0], m1 = tile_max[1], m2 = tile_max[2], m3 = tile_max[3];
                    odd = ((m0 | m1 | m2 | m3) >> 16) != 0u;
                    const uint32_t top = max(max(m0 & 0xffffu, m1 & 0xffffu), max(m2 & 0xffffu, m3 & 0xffffu));
                    const int k = fp16_scale_exp(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
                    vs = pow2i(k);
                    if (helper == 0 && t == 0) maxes[4 + (ch & 3)] = pow2i(-k);
                    if (!(ok = group_sync(&bars[sync], ph))) break;  // the maxima are read
                }
                const uint32_t stage = s * LY::kStage;
#pragma unroll 1
                for (int qd = 0; qd * kQuarter < n; ++qd) {
                    if (GROW && (qd & 1) != helper) {  // (growth pass: whole chunks, so each group keeps to one slot)
                        ++quarters;
                        continue;
                    }
                    const int r = quarters & 1, past = n - (qd + 1) * kQuarter;  // tokens after this quarter
                    float wt[8];
                    if (past >= 0) {
                        const float f = expf(g * static_cast<float>(past));
#pragma unroll
                        for (int i = 0; i < 8; ++i) wt[i] = f * fall[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int left = n - 1 - (qd * kQuarter + 8 * (i >> 1) + 2 * (lane & 3) + (i & 1));
                            wt[i] = left >= 0 ? expf(g * static_cast<float>(left)) : 0.f;
                        }
                    }
                    if constexpr (!BF) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) wt[i] *= vs;
                    }
                    uint32_t v[2][8];
                    if (live) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            ldmatrix_x4_trans(at[hh] + stage + qd * kQuarter * 128, v[hh]);
                            ldmatrix_x4_trans(at[hh] + stage + (qd * kQuarter + 16) * 128, v[hh] + 4);
                        }
                    }
                    if (quarters >= 2 && !(ok = mbar_wait_bounded(&bars[kVFree0 + r], ((quarters >> 1) - 1) & 1))) break;
                    ++quarters;
                    tc_fence_after();
                    if (live) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            float x[8], y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float2 f = unpack2<BF>(v[hh][i]);
                                x[i] = f.x * wt[2 * (i >> 1)];
                                y[i] = f.y * wt[2 * (i >> 1) + 1];
                            }
#pragma unroll
                            for (int q = 0; q < kParts; ++q) {
                                uint32_t part[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) part[i] = split2<BF>(x[i], y[i]);
                                tmem_st_16x128b_x4(tmem + (static_cast<uint32_t>(32 * w + 16 * hh) << 16) + kColV + r * kRing + 16 * q, part);
                            }
                        }
                        if constexpr (BF && !GROW) {
                            uint32_t zeros[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                            for (int i = 0; i < 16; ++i) add_zero_times(zeros[i & 3], v[i >> 3][i & 7]);
                            odd = odd || __any_sync(0xffffffffu, ((zeros[0] | zeros[1] | zeros[2] | zeros[3]) & 0x7fff7fffu) != 0u);
                        }
                        tmem_wait_st();
                        if (!GROW && __builtin_expect(odd && past <= 0, 0)) {  // (the warp has read all of its values)
                            const int dim = 32 * w + lane, slot = ch & 3;
                            first_odd[slot * 128 + dim] = static_cast<unsigned char>(take_out<BF>(sK + LY::kKBytes, dim, n));
                            if (lane == 0) odd_chunk[4 * slot + w] = ch;
                        }
                    }
                    tc_fence_before();
                    mbar_arrive(&bars[kVFull0 + r]);
                }
                if (!ok) break;
                mbar_arrive(&bars[kFree0 + s]);
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) flag(p.status, kDevTimeout);
            *abort_flag = 1;
        }
    };

    // The launch gives every thread 128 registers (4 x 128 in all); the groups
    // take 120, 216 and 96 (fp16, whose rows have their power of two besides: 128,
    // 208 and 96), which leaves 80 for the last: no spills.
    constexpr int kRowRegs = BF ? 120 : 128, kStateRegs = BF ? 216 : 208;
    if (warp == 13) {
        registers<80>();
        // ---------------- units and loads ----------------
        if (lane == 0) {
            int nu = 0, ch = 0, nq = 0;  // units published, chunks loaded (K and V, Q)
            const int vpanels = p.P > 64 ? 2 : 1;
            const int64_t units = (plan.head ? plan.head->pieces : p.nseq) * p.H;
            int64_t u = blockIdx.x;
            const auto next_unit = [&] {
                Unit un;
                for (;;) {
                    const int64_t now = u;
                    if (now >= units) {
                        un.len = -1;
                        return un;
                    }
                    u = plan.head ? atomicAdd(&plan.head->next[GROW ? 0 : 1], 1) : u + gridDim.x;
                    const int64_t b = now / p.H;
                    if (plan.head) {
                        un = plan.pieces[b];
                        if (GROW && un.h == 0) continue;
                    } else if (!find_sequence(p, b, un)) {
                        continue;
                    }
                    un.h = static_cast<int>(now - b * p.H);
                    return un;
                }
            };
            const auto publish = [&](const Unit &un) {
                // its first state on the way to L2
                if (!GROW && un.len >= 0 && un.src != kZero) {
                    const bool scratch = un.src >= kScratch;
                    const int64_t head = static_cast<int64_t>(p.P) * p.N, size = scratch || p.state_dtype == kF32 ? 4 : 2;
                    const unsigned char *state = scratch ? reinterpret_cast<const unsigned char *>(plan.states)
                                                         : static_cast<const unsigned char *>(p.state);
                    bulk_prefetch(state + ((scratch ? un.src - kScratch : un.src) * p.H + un.h) * head * size,
                                  static_cast<uint32_t>(head * size));
                }
                if (nu >= 2 && !mbar_wait_bounded(&bars[kUnitFree0 + (nu & 1)], ((nu >> 1) - 1) & 1)) return false;
                ring[nu & 1] = un;
                mbar_arrive(&bars[kUnitFull0 + (nu & 1)]);
                ++nu;
                return true;
            };
            // a unit is announced before the one ahead of it is loaded
            Unit un = next_unit();
            ok = publish(un);
            while (ok && un.len >= 0) {
                const Unit after = next_unit();
                if (!(ok = publish(after))) break;
                const int g = un.h / p.share;
                for (int c = 0; c < un.len; c += kC, ++ch) {
                    const int s = ch & 1, row = static_cast<int>(un.t0) + c;
                    if (ch >= 2 && !(ok = mbar_wait_bounded(&bars[kFree0 + s], ((ch >> 1) - 1) & 1))) break;
                    if (*abort_flag) ok = false;
                    if (!ok) break;
                    unsigned char *st = smem + s * LY::kStage;
                    mbar_arrive_expect(&bars[kFull0 + s], LY::kKBytes + vpanels * kPanel);
                    for (int i = 0; i < LY::kPanels; ++i)
                        tma_load_3d(st + i * kPanel, &maps.k, 64 * i, g, row, &bars[kFull0 + s]);
                    for (int i = 0; i < vpanels; ++i)
                        tma_load_3d(st + LY::kKBytes + i * kPanel, &maps.v, 64 * i, g, row, &bars[kFull0 + s]);
                    if constexpr (GROW) continue;
                    if (ch >= 2 && !(ok = mbar_wait_bounded(&bars[kQFree0 + s], ((ch >> 1) - 1) & 1))) {
                        ++ch;  // its K and V are on their way
                        break;
                    }
                    ++nq;
                    mbar_arrive_expect(&bars[kQFull0 + s], LY::kKBytes);
                    for (int i = 0; i < LY::kPanels; ++i)
                        tma_load_3d(smem + LY::kQ + s * LY::kQBytes + i * kPanel, &maps.q, 64 * i, un.h, row, &bars[kQFull0 + s]);
                }
                if (!ok) break;
                un = after;
            }
            if (!ok) {
                flag(p.status, kDevTimeout);
                *abort_flag = 1;
            }
            // what was loaded has landed before the CTA retires
            for (int k = ch > 2 ? ch - 2 : 0; k < ch; ++k) mbar_wait_bounded(&bars[kFull0 + (k & 1)], (k >> 1) & 1);
            for (int k = nq > 2 ? nq - 2 : 0; k < nq; ++k) mbar_wait_bounded(&bars[kQFull0 + (k & 1)], (k >> 1) & 1);
        }
        __syncwarp();
    } else if (warp == 12) {
        registers<80>();
        // ---------------- products (the warp together, one lane issuing) ----------------
        // Loop counts and addresses are the same in every lane and known to be
        // (shuffled from lane 0), so that descriptors stay in uniform registers:
        // formed per lane, each would be moved there again for every product.
        constexpr int bf = BF ? 1 : 0;
        const int ksteps = (p.N + 15) / 16, dims = (p.P + 15) / 16 * 16;
        const uint32_t id_score = idesc_f16(128, 128, 0, 0, bf), id_enter = idesc_f16(128, dims, 0, 0, bf);
        const uint32_t id_inside = idesc_f16(128, dims, 0, 1, bf), id_growth = idesc_f16(128, 16 * ksteps, 0, 1, bf);
        const uint32_t s0 = smem_addr(smem), tm = __shfl_sync(0xffffffffu, tmem, 0);
        const Desc dK(desc_k_sw128(s0)), dQ(desc_k_sw128(s0 + LY::kQ)), dS(desc_k_sw128(s0 + LY::kS));
        const Desc dKt(desc_mn_sw128(s0, kPanel)), dV(desc_mn_sw128(s0 + LY::kKBytes, kPanel));
        constexpr auto along_k = [](int k) { return static_cast<uint32_t>(((k / 4) * kPanel + (k % 4) * 32) >> 4); };
        constexpr auto along_mn = [](int k) { return static_cast<uint32_t>((k * 2048) >> 4); };
        const auto wait = [&](int bar, int phase) {
            const bool got = __all_sync(0xffffffffu, mbar_wait_bounded(&bars[bar], phase & 1));
            tc_fence_after();
            return got;
        };
        int nu = 0, quarters = 0;
        uint32_t tails = 0;  // bit s: phase of stage s's partial chunks
        struct Chunk {
            int ch, s, n, steps;  // running number, stage, tokens (0: no more), of them in 16s
            uint32_t stage;
        };
        int len = 0, c = 0, count = 0;  // the current unit's length, tokens begun, chunks begun
        const auto next_chunk = [&](Chunk &k) {
            while (c >= len) {
                if (!wait(kUnitFull0 + (nu & 1), nu >> 1)) return false;
                len = __shfl_sync(0xffffffffu, ring[nu & 1].len, 0);
                if (lane == 0) mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
                ++nu;
                c = 0;
                if (len < 0) {
                    k.n = 0;
                    return true;
                }
            }
            k.ch = count++;
            k.s = k.ch & 1;
            k.n = min(kC, len - c);
            k.steps = (k.n + 15) / 16;
            k.stage = static_cast<uint32_t>(k.s * (LY::kStage >> 4));
            c += kC;
            return true;
        };
        const auto growth = [&](const Chunk &k, int qd) {  // quarter qd, if there is one
            if (qd * kQuarter >= k.n) return true;
            if (qd == 0) {
                if (!wait(kFull0 + k.s, k.ch >> 1)) return false;
                if (k.n < kC) {
                    if (!wait(kTail0 + k.s, static_cast<int>(tails >> k.s))) return false;
                    tails ^= 1u << k.s;
                }
                if (k.ch > (GROW ? 1 : 0) && !wait(growth_free(k.ch), growth_phase(k.ch) - 1)) return false;
            }
            const int r = quarters & 1;
            if (!wait(kVFull0 + r, quarters >> 1)) return false;
            ++quarters;
            if (elect_one()) {
                const uint32_t a = tm + kColV + r * kRing;
                const Desc b = dKt + (k.stage + qd * along_mn(2));
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int part = 0; part < kParts; ++part)
                        if (2 * qd + i < k.steps)
                            mma_ts(tm + growth_at(k.ch), a + part * 16 + 8 * i, b + along_mn(i), id_growth, qd > 0 || i > 0 || part > 0);
                mma_commit(&bars[kVFree0 + r]);
                if ((qd + 1) * kQuarter >= k.n) {
                    mma_commit(&bars[growth_bar(k.ch)]);
                    if (GROW) mma_commit(&bars[kFree0 + k.s]);
                }
            }
            __syncwarp();
            return true;
        };
        // The quarters of the growth lie between the other products so that
        // each finds its decayed V prepared (two fit tensor memory at a time),
        // the scores become P meanwhile, and no product waits for the one
        // just before it.
        Chunk k;
        while ((ok = next_chunk(k)) && k.n > 0) {
            const uint32_t q = static_cast<uint32_t>(k.s * (LY::kQBytes >> 4));
            if (!(ok = growth(k, 0))) break;
            if constexpr (!GROW) {
                // (P of the last chunk, in the scores' place, has been read)
                if (!(ok = wait(kQFull0 + k.s, k.ch >> 1) && (k.ch == 0 || wait(kInside, k.ch - 1)))) break;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < DK / 16; ++i)
                        if (i < ksteps) mma(tm + kColScore, dQ + (q + along_k(i)), dK + (k.stage + along_k(i)), id_score, i > 0);
                    mma_commit(&bars[kScore]);
                }
                __syncwarp();
                if (!(ok = growth(k, 1))) break;
                if (!(ok = wait(kStateFull, k.ch) && (k.ch == 0 || wait(kOutFree, k.ch - 1)))) break;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < DK / 16; ++i)
                        if (i < ksteps) mma(tm + kColOut, dQ + (q + along_k(i)), dS + along_k(i), id_enter, i > 0);
                    mma_commit(&bars[kEnter]);
                }
                __syncwarp();
            }
            if (!(ok = (!GROW || growth(k, 1)) && growth(k, 2) && growth(k, 3))) break;
            if constexpr (!GROW) {
                if (!(ok = wait(kPFull, k.ch))) break;
                if (elect_one()) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < k.steps)
                            mma_ts(tm + kColOut, tm + kColScore + 8 * i, dV + (k.stage + along_mn(i)), id_inside, 1);
                    mma_commit(&bars[kInside]);
                    mma_commit(&bars[kFree0 + k.s]);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) {
            flag(p.status, kDevTimeout);
            *abort_flag = 1;
        }
        // every product issued has completed before tensor memory is freed
        if (elect_one()) mma_commit(&bars[kFinal]);
        __syncwarp();
        mbar_wait_bounded(&bars[kFinal], 0);
        __syncwarp();
    } else if (warp == 14) {
        registers<80>();
        // ---------------- output stores (one thread) ----------------
        if (!GROW && lane == 0) {
            int nu = 0, ch = 0;
            const int panels = p.P > 64 ? 2 : 1;
            for (;;) {
                if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
                const Unit un = ring[nu & 1];
                mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
                ++nu;
                if (un.len < 0) break;
                for (int c = 0; c < un.len; c += kC, ++ch) {
                    if (!(ok = mbar_wait_bounded(&bars[kStaged0 + (ch & 1)], (ch >> 1) & 1))) break;
                    if (un.len - c >= kC) {  // (a partial chunk's rows are stored one by one)
                        for (int i = 0; i < panels; ++i)
                            tma_store_3d(&maps.out, smem + LY::kQ + (ch & 1) * LY::kQBytes + i * kPanel, 64 * i, un.h,
                                         static_cast<int>(un.t0) + c);
                        bulk_commit();
                        bulk_wait_read<0>();
                    }
                    mbar_arrive(&bars[kQFree0 + (ch & 1)]);
                }
                if (!ok) break;
            }
            bulk_wait_all();
            if (!ok) {
                flag(p.status, kDevTimeout);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else if (warp == 15) {
        registers<80>();
    } else if (warp < 4) {
        registers<kRowRegs>();
        if constexpr (GROW) decay_values(1);
        // ---------------- P and the outputs (thread = token) ----------------
        const int row = tid;
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        int nu = 0, ch = 0, ph = 0;
        while (!GROW) {
            if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
            const Unit un = ring[nu & 1];
            mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
            ++nu;
            if (un.len < 0) break;
            const float g = fmaxf(__ldg(p.log_decay + un.h), -1e30f);  // 0 * -inf is no power
            const float g2 = g * 1.4426950408889634f;
            const float enter = p.scale * expf(g * static_cast<float>(row + 1));
            float fall[32];  // l^(31 - jj): from a column of a block to the block's last
#pragma unroll
            for (int jj = 0; jj < 32; ++jj) fall[jj] = ex2(g2 * static_cast<float>(31 - jj));
            unsigned short *out = static_cast<unsigned short *>(p.out) + un.h * p.os[1] + un.t0 * p.os[0];
            for (int c = 0; c < un.len; c += kC, ++ch) {
                const int n = min(kC, un.len - c);
                if (!(ok = mbar_wait_bounded(&bars[kScore], ch & 1))) break;
                tc_fence_after();
                // Row i of P: scale l^(i-j) score for j <= i.  A block of 32
                // columns before the warp's rows factors through its last
                // column, both powers at most 1; the block on the diagonal
                // takes one power a score.
                float up = 1.f, down = 1.f;  // fp16: the row's power of two
                if constexpr (!BF) {
                    // from the largest score before its decay, which bounds
                    // the decayed ones: P stays in fp16's normal range down to
                    // 2^-27 of it (of the scores up to the row's own token: a
                    // later one may be any number or none)
                    float m = 0.f;
#pragma unroll 1
                    for (int b = 0; b <= warp; ++b) {
                        uint32_t r[32];
                        tmem_ld32(tmem + lanes + kColScore + 32 * b, r);
                        tmem_wait_ld();
                        const int last = b < warp ? 31 : lane;
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj)
                            if (jj <= last) m = fmaxf(m, fabsf(__uint_as_float(r[jj])));
                    }
                    // (not so far up that the entering product, scaled alike, could overflow)
                    const int k = min(fp16_scale_exp(m * fabsf(p.scale)), 40);
                    up = pow2i(k);
                    down = pow2i(-k);
                }
                const float scale_up = p.scale * up;
                const auto decayed = [&](int b, float *e) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kColScore + 32 * b, r);
                    tmem_wait_ld();
                    if (b < warp) {
                        const float f = scale_up * ex2(g2 * static_cast<float>(row - 32 * b - 31));
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) e[jj] = __uint_as_float(r[jj]) * (f * fall[jj]);
                    } else {
#pragma unroll
                        for (int jj = 0; jj < 32; ++jj) {
                            const float w = scale_up * ex2(g2 * static_cast<float>(max(lane - jj, 0)));
                            e[jj] = jj <= lane ? __uint_as_float(r[jj]) * w : 0.f;
                        }
                    }
                };
                // (block b of P takes columns whose scores, of block b / 2, are read)
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t pr[16];
                    if (b <= warp) {
                        float e[32];
                        decayed(b, e);
#pragma unroll
                        for (int jj = 0; jj < 16; ++jj)
                            pr[jj] = pack2<BF>(e[2 * jj], e[2 * jj + 1]);
                    } else {
#pragma unroll
                        for (int jj = 0; jj < 16; ++jj) pr[jj] = 0u;
                    }
                    tmem_st16(tmem + lanes + kColScore + 16 * b, pr);
                }
                // the entering product's row, scaled in its place
                if (!(ok = mbar_wait_bounded(&bars[kEnter], ch & 1))) break;
                tc_fence_after();
                const float f = enter * up;
                // (fp16: value dim p's state row was scaled; written before the
                // product that has just completed was issued)
                const float *rs = row_scale + (ch & 1) * 128;
#pragma unroll 1
                for (int b = 0; 32 * b < p.P; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kColOut + 32 * b, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int jj = 0; jj < 32; ++jj)
                        r[jj] = __float_as_uint(__uint_as_float(r[jj]) * (BF ? f : f * rs[32 * b + jj]));
                    tmem_st32(tmem + lanes + kColOut + 32 * b, r);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&bars[kPFull]);
                if (!(ok = mbar_wait_bounded(&bars[kInside], ch & 1))) break;
                tc_fence_after();
                // Outputs by token where Q was (its products are done), laid out
                // for a tiled copy: a thread's own row, 16 or 32 bytes at a
                // time, would touch 32 lines a store.
                unsigned char *rows = smem + LY::kQ + (ch & 1) * LY::kQBytes, *mine = rows + row * 128;
#pragma unroll 1
                for (int b = 0; 32 * b < p.P; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + kColOut + 32 * b, r);
                    tmem_wait_ld();
                    if (32 * b + 32 >= p.P) {
                        tc_fence_before();
                        mbar_arrive(&bars[kOutFree]);
                    }
#pragma unroll
                    for (int jj = 0; jj < 16; ++jj) {
                        float x = __uint_as_float(r[2 * jj]), y = __uint_as_float(r[2 * jj + 1]);
                        if constexpr (!BF) x *= down, y *= down;
                        r[jj] = pack2<BF>(x, y);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4 *>(mine + (b / 2) * kPanel + (((4 * (b % 2) + j) ^ (row & 7)) * 16)) =
                            make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                }
                const int4 odd = reinterpret_cast<const int4 *>(odd_chunk)[ch & 3];
                if (__builtin_expect(odd.x == ch || odd.y == ch || odd.z == ch || odd.w == ch, 0)) {
                    const unsigned char *first = first_odd + (ch & 3) * 128;
#pragma unroll 1
                    for (int dim = 0; dim < p.P; ++dim)
                        if (odd_chunk[4 * (ch & 3) + dim / 32] == ch && row >= first[dim])
                            *reinterpret_cast<unsigned short *>(rows + swizzled(row, dim)) = 0x7fff;
                }
                fence_proxy_async_smem();
                if (n < kC) {
                    // the rows past the end are other tokens'
                    if (!(ok = group_sync(&bars[kSyncA], ph))) break;
                    const int piece = tid & 15;  // 16 threads store a token's row
                    if (8 * piece < p.P) {
                        for (int i = tid >> 4; i < n; i += kGroup / 16)
                            *reinterpret_cast<uint4 *>(out + (c + i) * p.os[0] + 8 * piece) = *reinterpret_cast<const uint4 *>(
                                rows + (piece / 8) * kPanel + i * 128 + (((piece % 8) ^ (i & 7)) * 16));
                    }
                }
                mbar_arrive(&bars[kStaged0 + (ch & 1)]);
            }
            if (!ok) break;
        }
        if (!ok) {
            if (lane == 0) flag(p.status, kDevTimeout);
            *abort_flag = 1;
        }
    } else if (warp < 8) {
        registers<kStateRegs>();
        // ---------------- the state (thread = value dim) ----------------
        const int t = tid - kGroup, w = warp - 4;
        const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
        int nu = 0, ch = 0, ph = 0;
        float S[DK];
        if constexpr (!GROW && !BF) {
            // fp16 scales a row of S by its largest, and S takes in all DK
            // columns of the growth, of which the products write dstate,
            // rounded up to 16.  The others, with what an earlier kernel left
            // in them, are zeros from here on (leaving them out of every sum
            // instead takes 10 % longer: 242 us for 217, 32768 tokens x 32 heads).
            const uint32_t zeros[16] = {};
            for (int c = (p.N + 15) / 16 * 16; c < DK; c += 16) tmem_st16(tmem + lanes + kColGrowth + c, zeros);
            tmem_wait_st();
        }
        for (;;) {
            if (!(ok = mbar_wait_bounded(&bars[kUnitFull0 + (nu & 1)], (nu >> 1) & 1))) break;
            const Unit un = ring[nu & 1];
            mbar_arrive(&bars[kUnitFree0 + (nu & 1)]);
            ++nu;
            if (un.len < 0) break;
            const float g = fmaxf(__ldg(p.log_decay + un.h), -1e30f);
            const float lam_chunk = expf(g * static_cast<float>(kC));
            const int64_t slot = static_cast<int64_t>(p.H) * p.P * p.N, head = static_cast<int64_t>(un.h) * p.P * p.N;
#pragma unroll
            for (int i = 0; i < DK; ++i) S[i] = 0.f;
            // the entering state, by way of its place for the products (which
            // the last entering product has read)
            if (!GROW && ch > 0 && !(ok = mbar_wait_bounded(&bars[kEnter], (ch - 1) & 1))) break;
            if (!GROW && un.src != kZero) {
                const bool scratch = un.src >= kScratch;
                const int64_t at = (scratch ? un.src - kScratch : un.src) * slot + head;
                const void *src = scratch ? plan.states : p.state;
                unsigned char *const place = smem + LY::kS;
                if (scratch || p.state_dtype == kF32) {
                    const float *from = static_cast<const float *>(src) + at;
                    stage_in<float, DK>(from, place, p.P, p.N, 0, t);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    if (t < p.P) row_from<float, DK, 0>(place, t, p.N, S);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    if (p.N > DK / 2) stage_in<float, DK>(from, place, p.P, p.N, DK / 2, t);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    if (t < p.P) row_from<float, DK, DK / 2>(place, t, p.N, S);
                } else {
                    stage_in<__half, DK>(static_cast<const __half *>(src) + at, place, p.P, p.N, 0, t);  // any 16 bits
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    if (t < p.P) {
                        if (p.state_dtype == kBF16) row_from<__nv_bfloat16, DK, 0>(place, t, p.N, S);
                        else row_from<__half, DK, 0>(place, t, p.N, S);
                    }
                }
                if (!(ok = group_sync(&bars[kSyncB], ph))) break;
            }
            for (int c = 0; c < un.len; c += kC, ++ch) {
                const int n = min(kC, un.len - c);
                if constexpr (!GROW) {
                    // S rounded, once the last entering product has read its own
                    float sc = 1.f;
                    if constexpr (!BF) {
                        float m = 0.f;
#pragma unroll
                        for (int i = 0; i < DK; ++i) m = fmaxf(m, fabsf(S[i]));
                        const int k = fp16_scale_exp(m);
                        sc = pow2i(k);
                        row_scale[(ch & 1) * 128 + t] = pow2i(-k);
                    }
                    if (ch > 0 && !(ok = mbar_wait_bounded(&bars[kEnter], (ch - 1) & 1))) break;
                    unsigned char *srow = smem + LY::kS + t * 128;
#pragma unroll
                    for (int j = 0; j < DK / 8; ++j) {
                        uint32_t u[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) u[i] = pack2<BF>(S[8 * j + 2 * i] * sc, S[8 * j + 2 * i + 1] * sc);
                        *reinterpret_cast<uint4 *>(srow + (j / 8) * kPanel + (((j % 8) ^ (t & 7)) * 16)) =
                            make_uint4(u[0], u[1], u[2], u[3]);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&bars[kStateFull]);
                }
                if (!(ok = mbar_wait_bounded(&bars[growth_bar(ch)], growth_phase(ch) & 1))) break;
                tc_fence_after();
                const float lam = n == kC ? lam_chunk : expf(g * static_cast<float>(n));
                const float back = BF ? 1.f : maxes[4 + (ch & 3)];
#pragma unroll
                for (int b = 0; b < DK / 32; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tmem + lanes + growth_at(ch) + 32 * b, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) S[32 * b + i] = fmaf(S[32 * b + i], lam, BF ? __uint_as_float(r[i]) : __uint_as_float(r[i]) * back);
                }
                tc_fence_before();
                mbar_arrive(&bars[growth_free(ch)]);
            }
            if (!ok) break;
            if (GROW || un.dst != kNone) {
                // out the same way
                if (!GROW && ch > 0 && !(ok = mbar_wait_bounded(&bars[kEnter], (ch - 1) & 1))) break;
                const int64_t at = (GROW ? un.src - kScratch : un.dst) * slot + head;
                unsigned char *const place = smem + LY::kS;
                void *dst = GROW ? plan.states : p.state;
                if (GROW || p.state_dtype == kF32) {
                    float *to = static_cast<float *>(dst) + at;
                    row_to<float, DK, 0>(place, t, S);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    stage_out<float, DK>(to, place, p.P, p.N, 0, t);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    row_to<float, DK, DK / 2>(place, t, S);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    if (p.N > DK / 2) stage_out<float, DK>(to, place, p.P, p.N, DK / 2, t);
                } else {
                    if (p.state_dtype == kBF16) row_to<__nv_bfloat16, DK, 0>(place, t, S);
                    else row_to<__half, DK, 0>(place, t, S);
                    if (!(ok = group_sync(&bars[kSyncB], ph))) break;
                    stage_out<__half, DK>(static_cast<__half *>(dst) + at, place, p.P, p.N, 0, t);
                }
                if (!(ok = group_sync(&bars[kSyncB], ph))) break;
            }
        }
        if (!ok) {
            if (lane == 0) flag(p.status, kDevTimeout);
            *abort_flag = 1;
        }
    } else {
        registers<96>();
        decay_values(0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tmem_dealloc512(tmem);
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
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

template <int DK, bool BF, bool GROW>
cudaError_t allow_smem() {
    return cudaFuncSetAttribute(linattn_prefill_kernel<DK, BF, GROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<DK>::kBytes);
}
template <int DK, bool BF, bool GROW>
cudaError_t launch_one(const LinattnParams &p, const Maps &maps, const Plan &plan, int64_t grid, cudaStream_t stream) {
    linattn_prefill_kernel<DK, BF, GROW><<<static_cast<unsigned>(grid), kThreads, Layout<DK>::kBytes, stream>>>(p, maps, plan);
    return cudaGetLastError();
}

template <int DK, bool BF>
cudaError_t launch_t(const LinattnParams &p, const LinattnSplit &split, void *workspace, cudaStream_t stream) {
    // Before the maps: their encoder is a driver call and refuses a host thread
    // that has no context yet, which this one gives it.
    cudaError_t e = allow_smem<DK, BF, false>();
    if (e == cudaSuccess && split.max_cuts > 0) e = allow_smem<DK, BF, true>();
    if (e != cudaSuccess) return e;
    Maps maps;
    if (p.rows > 0 && !(encode(&maps.q, p, p.q, p.N, p.H, p.qs) && encode(&maps.k, p, p.k, p.N, p.G, p.ks) &&
                        encode(&maps.v, p, p.v, p.P, p.G, p.vs) && encode(&maps.out, p, p.out, p.P, p.H, p.os)))
        return cudaErrorInvalidValue;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    Plan plan{};
    int64_t grid = p.nseq * p.H < sms ? p.nseq * p.H : sms;
    if (split.bytes > 0) {
        unsigned char *w = static_cast<unsigned char *>(workspace);
        plan.head = reinterpret_cast<PlanHead *>(w);
        plan.cuts = reinterpret_cast<Cut *>(w + split.cuts);
        plan.pieces = reinterpret_cast<Unit *>(w + split.pieces);
        plan.states = reinterpret_cast<float *>(w + split.states);
        plan.cut_len = split.cut_len;
        plan.max_cuts = split.max_cuts;
        plan.max_states = split.max_states;
        grid = sms;
        linattn_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, plan, static_cast<int>(grid));
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (split.max_cuts > 0) {
            if ((e = launch_one<DK, BF, true>(p, maps, plan, grid, stream)) != cudaSuccess) return e;
            const dim3 blocks(static_cast<unsigned>((static_cast<int64_t>(p.P) * p.N + 1023) / 1024), static_cast<unsigned>(p.H),
                              static_cast<unsigned>(split.max_cuts));
            linattn_carry_kernel<<<blocks, 256, 0, stream>>>(p, plan);
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
    }
    return launch_one<DK, BF, false>(p, maps, plan, grid, stream);
}

}  // namespace

// How a call is split.  Without cuts a call takes as long as its longest
// sequence on one SM (2.8 us a chunk), or its share of the GPU, `even` chunks an
// SM; cut into pieces of about `even` chunks it takes those, the growth pass
// over them (nearly as long again) and three more launches, worth 15 chunks.
// Measured, one sequence of 128 x 128 bf16 heads, four to a head of keys, uncut and
// cut: 40001 tokens x 16 heads 879 and 186 us, 4096 x 16 97 and 49, 2048 x 16 52 and
// 44 (the rule leaves it whole), 1024 x 16 30 and 41, 4096 x 64 99 and 119,
// 16384 x 64 367 and 348.  kSms, not the device's count: the workspace's size and
// the launch have to agree on the split whatever device is current at either.
LinattnSplit linattn_split(int64_t rows, int64_t nseq, int64_t heads, int64_t dim, int64_t dstate, int64_t max_seqlen) {
    constexpr int64_t kSms = 152;
    constexpr int64_t kCutCost = 15;
    LinattnSplit s{};
    if (nseq == 0 || rows == 0) return s;
    const auto chunks = [](int64_t n) { return (n + kC - 1) / kC; };
    // without a hint: the only sequence, or twice the mean
    int64_t longest = max_seqlen > 0 ? max_seqlen : nseq == 1 ? rows : 2 * ((rows + nseq - 1) / nseq);
    if (longest > rows) longest = rows;
    const int64_t even = (chunks(rows) * heads + kSms - 1) / kSms;
    const bool cut = chunks(longest) > 2 * even + kCutCost;
    if (!cut && nseq * heads <= kSms) return s;  // a CTA each: nothing to order
    const auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    // pieces a little longer than even, so that their number stays within a
    // whole round of the SMs
    const int64_t piece = even + (even + 15) / 16;
    s.cut_len = cut ? kC * (piece < 4 ? 4 : piece) : (rows + kC - 1) / kC * kC;
    s.max_cuts = cut ? rows / s.cut_len : 0;
    if (s.max_cuts > nseq) s.max_cuts = nseq;
    if (s.max_cuts > 65535) s.max_cuts = 65535;
    // sum over cut sequences of ceil(len / cut_len) <= 2 rows / cut_len
    s.max_states = cut ? 2 * (rows / s.cut_len) : 0;
    const uint64_t states = static_cast<uint64_t>(s.max_states);
    s.cuts = up(sizeof(PlanHead));
    s.pieces = s.cuts + up(s.max_cuts * sizeof(Cut));
    s.states = s.pieces + up((nseq + states) * sizeof(Unit));
    s.bytes = s.states + up(states * heads * dim * dstate * sizeof(float));
    return s;
}

cudaError_t launch_linattn_prefill(const LinattnParams &p, const LinattnSplit &split, void *workspace, cudaStream_t stream) {
    const bool bf = p.io_dtype == kBF16;
    if (p.N <= 64) return bf ? launch_t<64, true>(p, split, workspace, stream) : launch_t<64, false>(p, split, workspace, stream);
    return bf ? launch_t<128, true>(p, split, workspace, stream) : launch_t<128, false>(p, split, workspace, stream);
}

}  // namespace ssu
