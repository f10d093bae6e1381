// ssu_paged_append.cu -- new tokens' keys and values into their pages, keys and
// queries rotated on the way.
//
// Token i of the n new ones of a sequence of length L has position
// pos = L - n + i.  The first `rotary` elements of a head are pairs (x, y) --
// elements (j, j + rotary / 2), or (2 j, 2 j + 1) -- turned by the angle
// a = pos inv_freq[j]:
//     x' = x cos a - y sin a,   y' = y cos a + x sin a
// in fp32, rounded once.  The angle is formed and whole turns are taken off it in
// 64 bits (positions reach millions, where fp32 angles are off by whole radians);
// what is left, in half turns within [-1, 1], is rounded to fp32, by 2^-25 at most
// (2^-23 of an angle), and its sine and cosine are off by a little more than their
// own rounding.  (Of half turns: sincosf, with a path for large angles, made 150 us
// of 146 below.)
//
// HBM-bound: q, k and v are read once and written once.  A CTA takes T rows; a
// thread's item is 32 bytes of one head, two 16-byte pieces that hold whole
// pairs.  The first items are asked for before the metadata, whose reads depend
// on one another (sequence, length, page).  32768 rows of 32 + 2 x 8 heads of 128:
// 146 us in a graph (150 launched one by one), 5.5 TB/s, 0.82 of the copy rate: eight rows are at work on an SM, for
// 5.5 us each, and registers hold no more (48 or 56 a thread spill: 183, 148 us).
#include "ssu_paged.cuh"

namespace ssu {

namespace {

constexpr int kItems = 4;  // of a thread at a time

template <bool BF>
__device__ __forceinline__ void unpack8(const uint4 &u, float *v) {
    if constexpr (BF) StateChunk<__nv_bfloat16>::unpack(u, v);
    else StateChunk<__half>::unpack(u, v);
}
template <bool BF>
__device__ __forceinline__ uint4 pack8(const float *v) {
    if constexpr (BF) return StateChunk<__nv_bfloat16>::pack(v);
    else return StateChunk<__half>::pack(v);
}

// Division by a small number, by its reciprocal rounded down (exact below 2^16).
struct Divider {
    uint32_t by, inverse;
    __device__ __forceinline__ explicit Divider(int n) : by(n), inverse(0xffffffffu / static_cast<uint32_t>(n)) {}
    __device__ __forceinline__ int divide(int n, int &rest) const {
        uint32_t q = __umulhi(static_cast<uint32_t>(n), inverse), r = static_cast<uint32_t>(n) - q * by;
        if (r >= by) ++q, r -= by;
        rest = static_cast<int>(r);
        return static_cast<int>(q);
    }
};

struct Item {
    const unsigned short *src;
    int token, head, a, b;  // b < 0: one piece only
    bool turn;
};

template <bool BF, int T, int kThreads>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendParams p) {
    __shared__ int seq_of[T], row_of[T];  // row of its page
    __shared__ int64_t pos_of[T], page_of_row[T];  // page -1: none
    __shared__ float2 turn_by[T][kPagedMaxDim / 2];
    const PagedParams &c = p.c;
    const int tid = threadIdx.x;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * T;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(T), c.rows - r0));
    const int qheads = c.out ? c.H : 0, heads = qheads + 2 * c.G, per = (c.D + 15) / 16;
    const int items = tokens * heads * per, half = p.rotary / 2;

    const Divider by_per(per), by_heads(heads);
    const auto item = [&](int i) {
        Item it;
        int u;
        it.token = by_heads.divide(by_per.divide(i, u), it.head);
        const int64_t row = r0 + it.token;
        if (it.head < qheads) it.src = static_cast<const unsigned short *>(c.q) + row * c.qs[0] + it.head * c.qs[1];
        else if (it.head < qheads + c.G)
            it.src = static_cast<const unsigned short *>(p.k) + row * p.kstr[0] + (it.head - qheads) * p.kstr[1];
        else it.src = static_cast<const unsigned short *>(p.v) + row * p.vstr[0] + (it.head - qheads - c.G) * p.vstr[1];
        it.turn = it.head < qheads + c.G && 16 * u < p.rotary;
        if (it.turn && !p.interleaved) it.a = 8 * u, it.b = half + 8 * u;
        else it.a = 16 * u, it.b = 16 * u + 8 < c.D ? 16 * u + 8 : -1;
        return it;
    };
    uint4 a[kItems], b[kItems];
    const auto fetch = [&](int base) {
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = base + j * kThreads + tid;
            if (i >= items) continue;
            const Item it = item(i);
            a[j] = ld_stream(it.src + it.a);
            if (it.b >= 0) b[j] = ld_stream(it.src + it.b);
        }
    };
    fetch(0);

    if (tid < T) seq_of[tid] = -1;
    __syncthreads();
    // (with a row each, a row's sequence is known)
    const bool each = c.cu == nullptr;
    for (int64_t s = each ? r0 + tid : tid; s < (each ? r0 + tokens : c.nseq); s += kThreads) {
        const Seq q = load_seq(c, s, each || blockIdx.x == 0);
        const int64_t from = max(q.t0, r0), to = min(q.t0 + q.n, r0 + tokens);
        for (int64_t t = from; t < to; ++t) {
            // (where sequences overlap, which the last check does not exclude, one of them has the token)
            if (atomicCAS(&seq_of[t - r0], -1, static_cast<int>(s)) != -1) {
                flag(c.status, kDevBadSeqlen);
                continue;
            }
            const int64_t pos = q.kv - q.n + (t - q.t0);
            pos_of[t - r0] = pos;
            row_of[t - r0] = pos < 0 ? 0 : static_cast<int>(pos) % c.page;
            page_of_row[t - r0] = pos < 0 ? -1 : page_of(c, s, static_cast<int32_t>(pos));
        }
    }
    __syncthreads();
    for (int i = tid; i < tokens * half; i += kThreads) {
        const int t = i / half, j = i - t * half;
        if (seq_of[t] < 0) continue;
        const double turns = static_cast<double>(pos_of[t]) * static_cast<double>(__ldg(p.inv_freq + j)) * 0.15915494309189535;
        float s, co;
        sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s, &co);
        turn_by[t][j] = make_float2(co, s);
    }
    __syncthreads();

    for (int base = 0; base < items; base += kItems * kThreads) {
        if (base > 0) fetch(base);
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = base + j * kThreads + tid;
            if (i >= items) continue;
            const Item it = item(i);
            if (seq_of[it.token] < 0) continue;
            unsigned short *dst;
            if (it.head < qheads) {
                dst = static_cast<unsigned short *>(c.out) + (r0 + it.token) * c.os[0] + it.head * c.os[1];
            } else {
                const int64_t page = page_of_row[it.token];
                if (page < 0) continue;
                const bool key = it.head < qheads + c.G;
                const int64_t *str = key ? c.ks : c.vs;
                dst = static_cast<unsigned short *>(key ? c.k_cache : c.v_cache) + page * str[0] +
                      row_of[it.token] * str[1] + (it.head - qheads - (key ? 0 : c.G)) * str[2];
            }
            if (it.turn) {
                float x[8], y[8];
                unpack8<BF>(a[j], x);
                unpack8<BF>(b[j], y);
                // pair k of the item: elements x[k], y[k], or neighbours
                const float2 *cs = &turn_by[it.token][p.interleaved ? it.a / 2 : it.a];
                if (p.interleaved) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = cs[k], g = cs[k + 4];
                        const float x0 = x[2 * k], x1 = x[2 * k + 1], y0 = y[2 * k], y1 = y[2 * k + 1];
                        x[2 * k] = x0 * f.x - x1 * f.y, x[2 * k + 1] = x1 * f.x + x0 * f.y;
                        y[2 * k] = y0 * g.x - y1 * g.y, y[2 * k + 1] = y1 * g.x + y0 * g.y;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 f = cs[k];
                        const float u = x[k], v = y[k];
                        x[k] = u * f.x - v * f.y, y[k] = v * f.x + u * f.y;
                    }
                }
                a[j] = pack8<BF>(x);
                b[j] = pack8<BF>(y);
            }
            *reinterpret_cast<uint4 *>(dst + it.a) = a[j];
            if (it.b >= 0) *reinterpret_cast<uint4 *>(dst + it.b) = b[j];
        }
    }
}

template <bool BF, int T, int THREADS>
cudaError_t launch_t(const AppendParams &p, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>((p.c.rows + T - 1) / T);
    paged_append_kernel<BF, T, THREADS><<<grid, THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}
// Few rows: one a CTA of 256 threads, so that as many SMs as possible take part
// (3 rows 3.3 us in a graph, 3.7 with 128 threads).  More: CTAs of 128 threads, as
// many rows as those hold in one turn, one at least: 32768 rows of 32 + 2 x 8 heads
// of 128 150 us with one row, 4 in two turns 168; CTAs of 256 threads and two rows
// 156 to 164 (all with sincosf).
template <bool BF>
cudaError_t launch_b(const AppendParams &p, cudaStream_t stream) {
    constexpr int kHeld = 128 * kItems;
    const int items = ((p.c.out ? p.c.H : 0) + 2 * p.c.G) * ((p.c.D + 15) / 16);
    if (p.c.rows <= 8 * device_sms()) return launch_t<BF, 1, 256>(p, stream);
    if (2 * items > kHeld) return launch_t<BF, 1, 128>(p, stream);
    return 4 * items <= kHeld ? launch_t<BF, 4, 128>(p, stream) : launch_t<BF, 2, 128>(p, stream);
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams &p, cudaStream_t stream) {
    return p.c.io_dtype == kBF16 ? launch_b<true>(p, stream) : launch_b<false>(p, stream);
}

}  // namespace ssu
