// ssu_api.cpp -- the C ABI of libssu (include/ssu.h): argument checks, error
// messages and kernel selection.  Nothing here touches device memory; each
// update call is exactly one kernel launch on the caller's stream.
#include "ssu.h"

#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "ssu_hybrid.h"
#include "ssu_internal.h"
#include "ssu_paged.h"
#include "ssu_ssd_params.h"
#include "ssu_verify.h"

namespace {

thread_local char g_err[512] = "";

ssu_status fail(ssu_status st, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return st;
}

ssu_status ok() { return SSU_OK; }

bool valid_dtype(int32_t d) { return d == SSU_F32 || d == SSU_F16 || d == SSU_BF16; }
bool valid_itype(int32_t t) { return t == SSU_I32 || t == SSU_I64; }

// dstate -> lanes per state row (16 elements per lane), or 0 if unsupported.
int lanes_for(int64_t dstate) {
    switch (dstate) {
    case 16: return 1;
    case 32: return 2;
    case 64: return 4;
    case 128: return 8;
    case 256: return 16;
    }
    return 0;
}

const char *unsupported_name(uint32_t bits) {
    if (bits & SSU_UNSUP_RAND_SEED) return "rand_seed (stochastic rounding is not implemented)";
    if (bits & SSU_UNSUP_STATE_SCALE) return "state_scale";
    if (bits & SSU_UNSUP_INTERMEDIATE) return "intermediate_states_buffer / indices / scales";
    if (bits & SSU_UNSUP_CACHE_STEPS) return "cache_steps != 0";
    if (bits & SSU_UNSUP_ALGORITHM) return "algorithm / backend other than 'auto'";
    return "an unknown argument";
}

ssu_status check_shape(int32_t state_dtype, int32_t io_dtype, int32_t dt_dtype, int64_t heads,
                       int64_t dim, int64_t dstate, int64_t groups, int *lanes) {
    if (!valid_dtype(state_dtype)) return fail(SSU_ERR_INVALID, "state_dtype %d is not an ssu_dtype", state_dtype);
    if (!valid_dtype(io_dtype)) return fail(SSU_ERR_INVALID, "io_dtype %d is not an ssu_dtype", io_dtype);
    if (!valid_dtype(dt_dtype)) return fail(SSU_ERR_INVALID, "dt_dtype %d is not an ssu_dtype", dt_dtype);
    if (heads <= 0 || dim <= 0 || dstate <= 0 || groups <= 0)
        return fail(SSU_ERR_INVALID, "heads, dim, dstate and groups must be positive (got %lld, %lld, %lld, %lld)",
                    (long long)heads, (long long)dim, (long long)dstate, (long long)groups);
    if (heads % groups != 0)
        return fail(SSU_ERR_INVALID, "heads (%lld) must be divisible by groups (%lld)", (long long)heads,
                    (long long)groups);
    if (heads > (1 << 30) || dim > (1 << 30))
        return fail(SSU_ERR_INVALID, "heads and dim must be below 2^30");
    *lanes = lanes_for(dstate);
    if (*lanes == 0)
        return fail(SSU_ERR_UNSUPPORTED, "dstate %lld is not supported (16, 32, 64, 128 or 256)", (long long)dstate);
    return SSU_OK;
}

ssu_status check_strides(const char *name, const int64_t *s) {
    for (int i = 0; i < 3; ++i)
        if (s[i] < 0) return fail(SSU_ERR_INVALID, "%s_stride[%d] is negative", name, i);
    return SSU_OK;
}

// A pointer that the device reads elements of `size` bytes through.
bool aligned(const void *q, int64_t size) { return reinterpret_cast<uintptr_t>(q) % size == 0; }
int64_t dtype_size(int32_t dtype) { return dtype == SSU_F32 ? 4 : 2; }
int64_t itype_size(int32_t type) { return type == SSU_I64 ? 8 : 4; }

ssu_status check_table(const char *name, const ssu_slot_table *t, ssu::SlotTab *out) {
    std::memset(out, 0, sizeof *out);
    if (t == nullptr || t->entries == nullptr) return SSU_OK;
    if (!valid_itype(t->type)) return fail(SSU_ERR_INVALID, "%s table: type %d is not an ssu_itype", name, t->type);
    if (t->mode != SSU_SLOTS_STRIDED && t->mode != SSU_SLOTS_PER_ROW)
        return fail(SSU_ERR_INVALID, "%s table: mode %d is not an ssu_slot_mode", name, t->mode);
    if (t->extent < 0) return fail(SSU_ERR_INVALID, "%s table: negative extent", name);
    if (t->s0 < 0 || t->s1 < 0) return fail(SSU_ERR_INVALID, "%s table: negative stride", name);
    if (!aligned(t->entries, itype_size(t->type)))
        return fail(SSU_ERR_INVALID, "%s table: entries must be aligned to their type", name);
    out->entries = t->entries;
    out->s0 = t->s0;
    out->s1 = t->s1;
    out->extent = t->extent;
    out->is_i64 = t->type == SSU_I64;
    out->per_row = t->mode == SSU_SLOTS_PER_ROW;
    return SSU_OK;
}

// Shared checks; fills everything in `kp` except the packed layout.
ssu_status prepare(const ssu_args *a, int64_t rows, const ssu_slot_table *read, const ssu_slot_table *dst,
                   ssu::KParams *kp, int *lanes) {
    if (a == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (a->unsupported != 0)
        return fail(SSU_ERR_UNSUPPORTED, "not implemented: %s", unsupported_name(a->unsupported));
    if (a->reserved0 != 0) return fail(SSU_ERR_INVALID, "reserved0 must be 0");
    ssu_status st = check_shape(a->state_dtype, a->io_dtype, a->dt_dtype, a->heads, a->dim, a->dstate,
                                a->groups, lanes);
    if (st != SSU_OK) return st;
    if (a->slots <= 0) return fail(SSU_ERR_INVALID, "slots must be positive");
    if (!a->state || !a->A) return fail(SSU_ERR_INVALID, "state and A must not be NULL");
    if (rows > 0 && (!a->x || !a->dt || !a->B || !a->C || !a->y))
        return fail(SSU_ERR_INVALID, "x, dt, B, C and y must not be NULL");
    if (reinterpret_cast<uintptr_t>(a->state) % 16 != 0)
        return fail(SSU_ERR_INVALID, "state must be 16-byte aligned");

    if (rows > 0 && (a->y == a->x || a->y == a->z || a->y == a->dt || a->y == a->B || a->y == a->C ||
                     a->y == a->state))
        return fail(SSU_ERR_INVALID, "y must not alias an input");
    if ((st = check_strides("x", a->x_stride)) || (st = check_strides("dt", a->dt_stride)) ||
        (st = check_strides("B", a->B_stride)) || (st = check_strides("C", a->C_stride)) ||
        (st = check_strides("z", a->z_stride)) || (st = check_strides("y", a->y_stride)))
        return st;
    std::memset(kp, 0, sizeof *kp);
    if ((st = check_table("read", read, &kp->rd)) || (st = check_table("destination", dst, &kp->wr)))
        return st;
    kp->slots = a->slots;
    kp->H = static_cast<int32_t>(a->heads);
    kp->P = static_cast<int32_t>(a->dim);
    kp->N = static_cast<int32_t>(a->dstate);
    kp->G = static_cast<int32_t>(a->groups);
    kp->heads_per_group = static_cast<int32_t>(a->heads / a->groups);
    kp->ptiles = static_cast<int32_t>((a->dim + ssu::kTileRows - 1) / ssu::kTileRows);
    kp->io_dtype = a->io_dtype;
    kp->dt_dtype = a->dt_dtype;
    kp->softplus = a->dt_softplus != 0;
    kp->disable = a->disable_state_update != 0;
    kp->pad = a->pad_slot_id;
    kp->state = a->state;
    kp->x = a->x;
    kp->dt = a->dt;
    kp->B = a->B;
    kp->C = a->C;
    kp->z = a->z;
    kp->A = a->A;
    kp->D = a->D;
    kp->dt_bias = a->dt_bias;
    kp->y = a->y;
    for (int i = 0; i < 3; ++i) {
        kp->xs[i] = a->x_stride[i];
        kp->dts[i] = a->dt_stride[i];
        kp->Bs[i] = a->B_stride[i];
        kp->Cs[i] = a->C_stride[i];
        kp->zs[i] = a->z_stride[i];
        kp->ys[i] = a->y_stride[i];
    }
    kp->status = a->d_status;
    kp->wait_cycles = ssu::kDefaultWaitCycles;
    kp->withhold_unit = -1;
    return SSU_OK;
}

bool aligned16(const void *q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; }

// Which small operands the packed kernel can stage with bulk copies: every
// row it copies (B, C: dstate values of one row and group; x, z, dt: up to 64
// dim rows of one row and head) starts on a 16-byte boundary and is a
// multiple of 16 bytes long.
int32_t packed_bulk_ops(const ssu_args *a) {
    const int64_t io = a->io_dtype == SSU_F32 ? 4 : 2, dts = a->dt_dtype == SSU_F32 ? 4 : 2;
    auto rows_ok = [](const void *base, const int64_t *st, int64_t sz, int64_t count) {
        return base != nullptr && aligned16(base) && st[2] == 1 && (st[0] * sz) % 16 == 0 && (st[1] * sz) % 16 == 0 &&
               (count * sz) % 16 == 0;
    };
    int32_t ops = 0;
    if (rows_ok(a->B, a->B_stride, io, a->dstate) && rows_ok(a->C, a->C_stride, io, a->dstate)) ops |= ssu::kBulkBC;
    if (rows_ok(a->x, a->x_stride, io, a->dim) && (a->z == nullptr || rows_ok(a->z, a->z_stride, io, a->dim)))
        ops |= ssu::kBulkXZ;
    if (rows_ok(a->dt, a->dt_stride, dts, a->dim)) ops |= ssu::kBulkDT;
    return ops;
}

// The kernels launch on the current device: a state pool that lives on
// another device would be addressed from the wrong one.  Checked right before
// a launch, after every host check.
ssu_status check_device(const void *state, const char *what = "the state") {
    int dev = -1;
    cudaPointerAttributes pa;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(SSU_ERR_CUDA, "no current CUDA device");
    if (cudaPointerGetAttributes(&pa, state) != cudaSuccess) {
        cudaGetLastError();
        return fail(SSU_ERR_INVALID, "the pointer of %s is not one the CUDA runtime knows", what);
    }
    if (pa.type == cudaMemoryTypeDevice && pa.device != dev)
        return fail(SSU_ERR_INVALID, "%s is on device %d but device %d is current", what, pa.device, dev);
    return SSU_OK;
}

ssu_status launched(cudaError_t e) {
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "kernel launch failed: %s", cudaGetErrorString(e));
    return ok();
}

constexpr int64_t kMaxGrid = 0x7fffffffLL;

}  // namespace

extern "C" {

ssu_status ssu_update_onetoken(const ssu_args *args, int64_t batch, const ssu_slot_table *read,
                               const ssu_slot_table *dst, void *stream) {
    ssu::KParams kp;
    int lanes = 0;
    if (batch < 0) return fail(SSU_ERR_INVALID, "batch is negative");
    ssu_status st = prepare(args, batch, read, dst, &kp, &lanes);
    if (st != SSU_OK) return st;
    if (batch == 0) return ok();
    if (batch * kp.H * kp.ptiles > kMaxGrid) return fail(SSU_ERR_INVALID, "batch * heads * dim tiles exceeds 2^31-1");
    kp.nseq = batch;
    kp.rows = batch;
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_onetoken(args->state_dtype, lanes, kp, batch,
                                         static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_selftest_timeout(const ssu_args *args, int64_t batch, const ssu_slot_table *read,
                                const ssu_slot_table *dst, int64_t withhold_unit, int64_t wait_cycles,
                                void *stream) {
    ssu::KParams kp;
    int lanes = 0;
    if (batch <= 0) return fail(SSU_ERR_INVALID, "batch must be positive");
    ssu_status st = prepare(args, batch, read, dst, &kp, &lanes);
    if (st != SSU_OK) return st;
    if (batch * kp.H * kp.ptiles > kMaxGrid) return fail(SSU_ERR_INVALID, "batch * heads * dim tiles exceeds 2^31-1");
    if (withhold_unit < 0 || withhold_unit >= batch * kp.H * kp.ptiles)
        return fail(SSU_ERR_INVALID, "withhold_unit must name a unit of the call");
    if (wait_cycles < 1000 || wait_cycles > ssu::kDefaultWaitCycles)
        return fail(SSU_ERR_INVALID, "wait_cycles must be in [1000, %lld]", (long long)ssu::kDefaultWaitCycles);
    kp.nseq = batch;
    kp.rows = batch;
    kp.withhold_unit = withhold_unit;
    kp.wait_cycles = wait_cycles;
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_onetoken(args->state_dtype, lanes, kp, batch, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_update_packed(const ssu_args *args, int64_t nseq, int64_t rows, const void *cu_seqlens,
                             int64_t steps, const void *num_accepted, int32_t meta_type,
                             const ssu_slot_table *read, const ssu_slot_table *dst, void *stream) {
    ssu::KParams kp;
    int lanes = 0;
    if (nseq < 0 || rows < 0) return fail(SSU_ERR_INVALID, "nseq and rows must not be negative");
    ssu_status st = prepare(args, rows, read, dst, &kp, &lanes);
    if (st != SSU_OK) return st;
    if ((cu_seqlens != nullptr || num_accepted != nullptr) && !valid_itype(meta_type))
        return fail(SSU_ERR_INVALID, "meta_type %d is not an ssu_itype", meta_type);
    if (cu_seqlens == nullptr) {
        if (steps <= 0) return fail(SSU_ERR_INVALID, "dense form (no cu_seqlens) needs steps > 0");
        if (rows != nseq * steps)
            return fail(SSU_ERR_INVALID, "dense form: rows (%lld) must equal nseq * steps (%lld)", (long long)rows,
                        (long long)(nseq * steps));
    }
    if (nseq == 0 || rows == 0) return ok();  // nothing to read or write
    if (nseq * kp.H * kp.ptiles > kMaxGrid) return fail(SSU_ERR_INVALID, "nseq * heads * dim tiles exceeds 2^31-1");
    if ((rows + nseq) > (int64_t(1) << 40) / (static_cast<int64_t>(kp.H) * kp.ptiles))
        return fail(SSU_ERR_INVALID, "(rows + nseq) * heads * dim tiles exceeds 2^40");
    kp.nseq = nseq;
    kp.rows = rows;
    kp.bulk_ops = packed_bulk_ops(args);
    kp.steps = cu_seqlens == nullptr ? steps : 0;
    kp.cu = cu_seqlens;
    kp.acc = num_accepted;
    kp.meta_is_i64 = meta_type == SSU_I64;
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_packed(args->state_dtype, lanes, kp, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_replay_update(const ssu_args *args, int64_t batch, const ssu_slot_table *slots,
                             const ssu_replay_buffers *rb, void *stream) {
    ssu::KParams kp;
    int lanes = 0;
    if (batch < 0) return fail(SSU_ERR_INVALID, "batch is negative");
    ssu_status st = prepare(args, batch, slots, nullptr, &kp, &lanes);
    if (st != SSU_OK) return st;
    if (args->disable_state_update) return fail(SSU_ERR_INVALID, "disable_state_update is not defined for the replay step");
    if (rb == nullptr) return fail(SSU_ERR_INVALID, "replay buffers are NULL");
    if (rb->len < 1 || rb->len > ssu::kMaxReplayLen)
        return fail(SSU_ERR_UNSUPPORTED, "buffer length %lld is not supported (1..%d)", (long long)rb->len,
                    ssu::kMaxReplayLen);
    if (batch == 0) return ok();
    if (!rb->x || !rb->dt || !rb->B || !rb->count_in || !rb->count_out)
        return fail(SSU_ERR_INVALID, "replay buffers and counts must not be NULL");
    if (rb->count_out == rb->count_in) return fail(SSU_ERR_INVALID, "count_out must not alias count_in");
    if (batch * kp.H * kp.ptiles > kMaxGrid) return fail(SSU_ERR_INVALID, "batch * heads * dim tiles exceeds 2^31-1");
    kp.nseq = batch;
    kp.rows = batch;
    kp.rlen = static_cast<int32_t>(rb->len);
    kp.xbuf = rb->x;
    kp.dtbuf = rb->dt;
    kp.Bbuf = rb->B;
    kp.cnt_in = rb->count_in;
    kp.cnt_out = rb->count_out;
    {
        const int64_t io = args->io_dtype == SSU_F32 ? 4 : 2;
        const bool aligned = reinterpret_cast<uintptr_t>(rb->x) % 16 == 0 && reinterpret_cast<uintptr_t>(rb->dt) % 16 == 0 &&
                             reinterpret_cast<uintptr_t>(rb->B) % 16 == 0;
        kp.rbulk = aligned && (args->dim * io) % 16 == 0 && (args->dim * 4) % 16 == 0 && (args->dstate * io) % 16 == 0;
    }
    if (rb->reserved0 != 0) return fail(SSU_ERR_INVALID, "replay buffers: reserved0 must be 0");
    kp.shadow_fmt = rb->shadow_format;
    if (rb->shadow_format != SSU_SHADOW_NONE) {
        if (rb->shadow_format != SSU_SHADOW_F16 && rb->shadow_format != SSU_SHADOW_E4M3 &&
            rb->shadow_format != SSU_SHADOW_NVFP4)
            return fail(SSU_ERR_INVALID, "shadow_format %d is not an SSU_SHADOW_* value", rb->shadow_format);
        if (rb->shadow == nullptr || reinterpret_cast<uintptr_t>(rb->shadow) % 16 != 0)
            return fail(SSU_ERR_INVALID, "the read copy must be a 16-byte aligned device pointer");
        if (rb->shadow_format == SSU_SHADOW_E4M3) {
            if (rb->shadow_scale == nullptr || reinterpret_cast<uintptr_t>(rb->shadow_scale) % 16 != 0)
                return fail(SSU_ERR_INVALID, "E4M3 row scales must be a 16-byte aligned device pointer");
            if (args->dim % 4 != 0)
                return fail(SSU_ERR_UNSUPPORTED, "an E4M3 read copy needs dim to be a multiple of 4");
        }
        if (rb->shadow_format == SSU_SHADOW_NVFP4) {
            if (rb->shadow_scale == nullptr || reinterpret_cast<uintptr_t>(rb->shadow_scale) % 16 != 0)
                return fail(SSU_ERR_INVALID, "NVFP4 scale records must be a 16-byte aligned device pointer");
            if (args->dstate != 64 && args->dstate != 128 && args->dstate != 256)
                return fail(SSU_ERR_UNSUPPORTED, "an NVFP4 read copy needs dstate 64, 128 or 256");
        }
        kp.shadow = rb->shadow;
        kp.shadow_scale = rb->shadow_scale;
    }
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_replay(args->state_dtype, lanes, kp, batch, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_replay_verify(const ssu_args *args, int64_t batch, int64_t ntok, const ssu_slot_table *slots,
                             const ssu_replay_buffers *rb, void *stream) {
    ssu::KParams kp;
    int lanes = 0;
    if (batch < 0) return fail(SSU_ERR_INVALID, "batch is negative");
    if (ntok < 1) return fail(SSU_ERR_INVALID, "ntok must be at least 1");
    ssu_status st = prepare(args, batch * ntok, slots, nullptr, &kp, &lanes);
    if (st != SSU_OK) return st;
    if (args->disable_state_update) return fail(SSU_ERR_INVALID, "disable_state_update is not defined for verification");
    if (rb == nullptr) return fail(SSU_ERR_INVALID, "replay buffers are NULL");
    if (rb->len < 1 || rb->len > ssu::kMaxReplayLen)
        return fail(SSU_ERR_UNSUPPORTED, "buffer length %lld is not supported (1..%d)", (long long)rb->len,
                    ssu::kMaxReplayLen);
    if (ntok > rb->len) return fail(SSU_ERR_INVALID, "ntok (%lld) exceeds the buffer length (%lld)", (long long)ntok,
                                    (long long)rb->len);
    if (rb->reserved0 != 0) return fail(SSU_ERR_INVALID, "replay buffers: reserved0 must be 0");
    if (rb->shadow_format != SSU_SHADOW_NONE)
        return fail(SSU_ERR_UNSUPPORTED, "verification does not read a low-precision copy");
    if (batch == 0) return ok();
    if (!rb->x || !rb->dt || !rb->B || !rb->count_in || !rb->count_out)
        return fail(SSU_ERR_INVALID, "replay buffers and counts must not be NULL");
    if (rb->count_out == rb->count_in) return fail(SSU_ERR_INVALID, "count_out must not alias count_in");
    if (args->heads > 65535 || batch > kMaxGrid || (args->dim + 63) / 64 > 65535)
        return fail(SSU_ERR_INVALID, "too many heads, sequences or dim rows for one launch");
    kp.nseq = batch;
    kp.rows = batch * ntok;
    kp.rlen = static_cast<int32_t>(rb->len);
    kp.xbuf = rb->x;
    kp.dtbuf = rb->dt;
    kp.Bbuf = rb->B;
    kp.cnt_in = rb->count_in;
    kp.cnt_out = rb->count_out;
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_verify(args->state_dtype, kp, batch, static_cast<int>(ntok),
                                       static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_batch_copy(const ssu_copy *copies, int64_t n, uint64_t max_bytes, int32_t *d_status,
                          void *stream) {
    if (n < 0) return fail(SSU_ERR_INVALID, "n is negative");
    if (n == 0 || max_bytes == 0) return ok();
    if (copies == nullptr) return fail(SSU_ERR_INVALID, "copies is NULL");
    if (reinterpret_cast<uintptr_t>(copies) % 8 != 0) return fail(SSU_ERR_INVALID, "copies must be 8-byte aligned");
    if (d_status != nullptr && reinterpret_cast<uintptr_t>(d_status) % 4 != 0)
        return fail(SSU_ERR_INVALID, "d_status must be 4-byte aligned");
    return launched(ssu::launch_copy(copies, n, max_bytes, d_status, static_cast<cudaStream_t>(stream)));
}

// Workspace carve-up of the SSD prefill: chunk states, prefix sums, dt',
// chunk decays, the largest |x| and dt' per (chunk, head); each part
// 256-byte aligned.
struct SsdWorkspace {
    uint64_t state, acs, dtp, dec, scl, total;
};
static SsdWorkspace ssd_workspace(uint64_t nchunks, uint64_t heads, uint64_t dim, uint64_t dstate,
                                  uint64_t chunk_size) {
    auto up = [](uint64_t v) { return (v + 255) / 256 * 256; };
    const uint64_t ch = nchunks * heads;
    SsdWorkspace w{};
    w.state = 0;
    w.acs = w.state + up(ch * dim * dstate * 4);
    w.dtp = w.acs + up(ch * chunk_size * 4);
    w.dec = w.dtp + up(ch * chunk_size * 4);
    w.scl = w.dec + up(ch * 4);
    w.total = w.scl + up(ch * 16);
    return w;
}

ssu_status ssu_ssd_workspace_size(int64_t nchunks, int64_t heads, int64_t groups, int64_t dim, int64_t dstate,
                                  int64_t chunk_size, uint64_t *bytes) {
    if (!bytes) return fail(SSU_ERR_INVALID, "bytes is NULL");
    if (nchunks < 0 || heads <= 0 || groups <= 0 || dim <= 0 || dstate <= 0 || chunk_size <= 0)
        return fail(SSU_ERR_INVALID, "sizes must be positive (nchunks >= 0)");
    *bytes = ssd_workspace(nchunks, heads, dim, dstate, chunk_size).total;
    return ok();
}

ssu_status ssu_ssd_prefill(const ssu_ssd_args *a, void *stream) {
    if (a == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (a->tokens < 0 || a->nseq < 0 || a->nchunks < 0) return fail(SSU_ERR_INVALID, "negative sizes");
    if (a->heads <= 0 || a->groups <= 0 || a->heads % a->groups != 0)
        return fail(SSU_ERR_INVALID, "heads (%lld) must be a positive multiple of groups (%lld)", (long long)a->heads,
                    (long long)a->groups);
    if (a->io_dtype != SSU_BF16) return fail(SSU_ERR_UNSUPPORTED, "the SSD prefill takes bf16 x, z, B, C and y");
    if (!valid_dtype(a->dt_dtype) || !valid_dtype(a->state_dtype)) return fail(SSU_ERR_INVALID, "bad dtype");
    if (!valid_itype(a->meta_type)) return fail(SSU_ERR_INVALID, "meta_type %d is not an ssu_itype", a->meta_type);
    if (a->dim != 64) return fail(SSU_ERR_UNSUPPORTED, "the SSD prefill supports dim 64 (got %lld)", (long long)a->dim);
    if (a->dstate != 64 && a->dstate != 128)
        return fail(SSU_ERR_UNSUPPORTED, "the SSD prefill supports dstate 64 or 128 (got %lld)", (long long)a->dstate);
    if (a->chunk_size != 64 && a->chunk_size != 128 && a->chunk_size != 256)
        return fail(SSU_ERR_UNSUPPORTED, "chunk_size %lld is not supported (64, 128, 256)", (long long)a->chunk_size);
    if (!(a->dt_min <= a->dt_max)) return fail(SSU_ERR_INVALID, "dt_limit must satisfy min <= max");
    if (a->nchunks == 0 || a->tokens == 0) return ok();
    if (a->nchunks > 65535 || a->heads > 65535) return fail(SSU_ERR_INVALID, "more than 65535 chunks or heads");
    if (!a->x || !a->dt || !a->B || !a->C || !a->A || !a->cu_chunk_seqlens || !a->seq_idx || !a->y || !a->states ||
        (!a->return_intermediate && !a->last_chunk_indices) || !a->workspace)
        return fail(SSU_ERR_INVALID, "a required pointer is NULL");
    const void *aligned[] = {a->x, a->B, a->C, a->y, a->states, a->workspace, a->z, a->initial_states};
    for (const void *q : aligned)
        if (reinterpret_cast<uintptr_t>(q) % 16 != 0) return fail(SSU_ERR_INVALID, "tensors must be 16-byte aligned");
    const SsdWorkspace wl = ssd_workspace(a->nchunks, a->heads, a->dim, a->dstate, a->chunk_size);
    const uint64_t need = wl.total;
    if (a->workspace_bytes < need)
        return fail(SSU_ERR_INVALID, "workspace of %lld bytes is smaller than the %lld needed",
                    (long long)a->workspace_bytes, (long long)need);
    ssu::SsdParams p{};
    p.tokens = a->tokens;
    p.nchunks = a->nchunks;
    p.nseq = a->nseq;
    p.H = static_cast<int32_t>(a->heads);
    p.G = static_cast<int32_t>(a->groups);
    p.hpg = static_cast<int32_t>(a->heads / a->groups);
    p.P = static_cast<int32_t>(a->dim);
    p.N = static_cast<int32_t>(a->dstate);
    p.Q = static_cast<int32_t>(a->chunk_size);
    p.dt_dtype = a->dt_dtype;
    p.state_dtype = a->state_dtype;
    p.softplus = a->dt_softplus != 0;
    p.intermediate = a->return_intermediate != 0;
    p.meta_i64 = a->meta_type == SSU_I64;
    p.dt_lo = a->dt_min;
    p.dt_hi = a->dt_max;
    p.x = a->x, p.dt = a->dt, p.B = a->B, p.C = a->C, p.z = a->z;
    p.A = a->A, p.D = a->D, p.dt_bias = a->dt_bias;
    p.cu_chunk = a->cu_chunk_seqlens, p.seq_idx = a->seq_idx, p.last_chunk = a->last_chunk_indices;
    p.init = a->initial_states;
    p.y = a->y;
    p.states = a->states;
    p.status = a->d_status;
    {
        unsigned char *w = static_cast<unsigned char *>(a->workspace);
        p.ws_state = reinterpret_cast<float *>(w + wl.state);
        p.ws_acs = reinterpret_cast<float *>(w + wl.acs);
        p.ws_dtp = reinterpret_cast<float *>(w + wl.dtp);
        p.ws_dec = reinterpret_cast<float *>(w + wl.dec);
        p.ws_scl = reinterpret_cast<float *>(w + wl.scl);
    }
    return launched(ssu::launch_ssd(p, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_ssd_prefill_static(const ssu_ssd_args *args, void *stream) {
    if (args == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (args->workspace != nullptr || args->workspace_bytes != 0)
        return fail(SSU_ERR_INVALID, "workspace must be NULL and workspace_bytes 0 (the library's scratch is used)");
    uint64_t need = 0;
    const ssu_status st = ssu_ssd_workspace_size(args->nchunks, args->heads, args->groups, args->dim, args->dstate,
                                                 args->chunk_size, &need);
    if (st != SSU_OK) return st;
    if (need > ssu::kSsdStaticScratchBytes)
        return fail(SSU_ERR_INVALID, "the call needs %llu bytes of workspace; the library's scratch holds %llu",
                    (unsigned long long)need, (unsigned long long)ssu::kSsdStaticScratchBytes);
    if (args->nchunks == 0 || args->tokens == 0) return ssu_ssd_prefill(args, stream);
    void *scratch = nullptr;
    const cudaError_t e = ssu::ssd_static_scratch(&scratch);
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "looking up the scratch failed: %s", cudaGetErrorString(e));
    ssu_ssd_args a = *args;
    a.workspace = scratch;
    a.workspace_bytes = ssu::kSsdStaticScratchBytes;
    return ssu_ssd_prefill(&a, stream);
}

ssu_status ssu_shadow_refresh(const void *state, int32_t state_dtype, int64_t rows, int64_t dstate,
                              int32_t format, void *shadow, float *scale, void *stream) {
    if (!valid_dtype(state_dtype)) return fail(SSU_ERR_INVALID, "state_dtype %d is not an ssu_dtype", state_dtype);
    if (format != SSU_SHADOW_F16 && format != SSU_SHADOW_E4M3 && format != SSU_SHADOW_NVFP4)
        return fail(SSU_ERR_INVALID, "format %d is not SSU_SHADOW_F16, SSU_SHADOW_E4M3 or SSU_SHADOW_NVFP4", format);
    if (rows < 0 || dstate <= 0 || dstate > 4096) return fail(SSU_ERR_INVALID, "rows must be >= 0, dstate in [1, 4096]");
    if (format == SSU_SHADOW_NVFP4 && dstate % 32 != 0)
        return fail(SSU_ERR_UNSUPPORTED, "an NVFP4 read copy needs dstate to be a multiple of 32");
    if (rows == 0) return ok();
    if (!state || !shadow || (format != SSU_SHADOW_F16 && !scale))
        return fail(SSU_ERR_INVALID, "state, shadow (and scale for E4M3 and NVFP4) must not be NULL");
    return launched(ssu::launch_shadow_refresh(state, state_dtype, rows, static_cast<int>(dstate), format, shadow,
                                               scale, static_cast<cudaStream_t>(stream)));
}

// Checks shared by the two forms of linear attention; fills `lp` except the
// packed layout.
static ssu_status linattn_prepare(const ssu_linattn_args *a, const ssu_slot_table *read, const ssu_slot_table *dst,
                                  ssu::LinattnParams *lp) {
    if (a == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (a->reserved0 != 0) return fail(SSU_ERR_INVALID, "reserved0 must be 0");
    if (!valid_dtype(a->io_dtype)) return fail(SSU_ERR_INVALID, "io_dtype %d is not an ssu_dtype", a->io_dtype);
    if (!valid_dtype(a->state_dtype))
        return fail(SSU_ERR_INVALID, "state_dtype %d is not an ssu_dtype", a->state_dtype);
    if (a->rows < 0) return fail(SSU_ERR_INVALID, "rows is negative");
    if (a->slots <= 0) return fail(SSU_ERR_INVALID, "slots must be positive");
    if (a->heads <= 0 || a->kv_heads <= 0 || a->heads % a->kv_heads != 0)
        return fail(SSU_ERR_INVALID, "heads (%lld) must be a positive multiple of kv_heads (%lld)", (long long)a->heads,
                    (long long)a->kv_heads);
    if (a->heads > 65535) return fail(SSU_ERR_INVALID, "more than 65535 heads");
    for (const int64_t d : {a->dim, a->dstate})
        if (d < 8 || d > ssu::kLinattnMaxDim || d % 8 != 0)
            return fail(SSU_ERR_UNSUPPORTED, "dim %lld, dstate %lld: linear attention takes multiples of 8 from 8 to %d",
                        (long long)a->dim, (long long)a->dstate, ssu::kLinattnMaxDim);
    if (!(a->scale == a->scale)) return fail(SSU_ERR_INVALID, "scale is not a number");
    if (!a->state || !a->log_decay) return fail(SSU_ERR_INVALID, "state and log_decay must not be NULL");
    if (!aligned16(a->state)) return fail(SSU_ERR_INVALID, "state must be 16-byte aligned");
    for (const void *q : {a->q, a->k, a->v, static_cast<const void *>(a->out)})
        if (!aligned(q, dtype_size(a->io_dtype))) return fail(SSU_ERR_INVALID, "q, k, v and out must be aligned to their type");
    if (!aligned(a->log_decay, 4) || !aligned(a->d_status, 4))
        return fail(SSU_ERR_INVALID, "log_decay and d_status must be 4-byte aligned");
    if (a->rows > 0 && (!a->q || !a->k || !a->v || !a->out)) return fail(SSU_ERR_INVALID, "q, k, v and out must not be NULL");
    if (a->rows > 0 && (a->out == a->q || a->out == a->k || a->out == a->v || a->out == a->state))
        return fail(SSU_ERR_INVALID, "out must not alias an input");
    std::memset(lp, 0, sizeof *lp);
    for (int i = 0; i < 2; ++i) {
        if (a->q_stride[i] < 0 || a->k_stride[i] < 0 || a->v_stride[i] < 0 || a->out_stride[i] < 0)
            return fail(SSU_ERR_INVALID, "a stride is negative");
        lp->qs[i] = a->q_stride[i], lp->ks[i] = a->k_stride[i], lp->vs[i] = a->v_stride[i], lp->os[i] = a->out_stride[i];
    }
    ssu_status st;
    if ((st = check_table("read", read, &lp->rd)) || (st = check_table("destination", dst, &lp->wr))) return st;
    // a table has one entry per sequence, (b, 0): the mode is ignored
    lp->rd.per_row = lp->wr.per_row = 0;
    lp->slots = a->slots;
    lp->rows = a->rows;
    lp->H = static_cast<int32_t>(a->heads);
    lp->G = static_cast<int32_t>(a->kv_heads);
    lp->share = static_cast<int32_t>(a->heads / a->kv_heads);
    lp->P = static_cast<int32_t>(a->dim);
    lp->N = static_cast<int32_t>(a->dstate);
    lp->io_dtype = a->io_dtype;
    lp->state_dtype = a->state_dtype;
    lp->scale = a->scale;
    lp->pad = a->pad_slot_id;
    lp->state = a->state;
    lp->q = a->q, lp->k = a->k, lp->v = a->v;
    lp->log_decay = a->log_decay;
    lp->out = a->out;
    lp->status = a->d_status;
    return SSU_OK;
}

ssu_status ssu_linear_attention_step(const ssu_linattn_args *args, const ssu_slot_table *read,
                                     const ssu_slot_table *dst, void *stream) {
    ssu::LinattnParams lp;
    ssu_status st = linattn_prepare(args, read, dst, &lp);
    if (st != SSU_OK) return st;
    if (lp.rows == 0) return ok();
    if (lp.rows > kMaxGrid / (4 * lp.H)) return fail(SSU_ERR_INVALID, "too many sequences and heads for one launch");
    lp.nseq = lp.rows;
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_linattn_step(lp, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_linear_attention_workspace_size(const ssu_linattn_args *args, int64_t nseq, int64_t max_seqlen,
                                               uint64_t *bytes) {
    if (!bytes) return fail(SSU_ERR_INVALID, "bytes is NULL");
    if (nseq < 0 || max_seqlen < 0) return fail(SSU_ERR_INVALID, "nseq and max_seqlen must not be negative");
    ssu::LinattnParams lp;
    const ssu_status st = linattn_prepare(args, nullptr, nullptr, &lp);
    if (st != SSU_OK) return st;
    *bytes = ssu::linattn_split(lp.rows, nseq, lp.H, lp.P, lp.N, max_seqlen).bytes;
    return ok();
}

ssu_status ssu_linear_attention_prefill(const ssu_linattn_args *args, int64_t nseq, const void *cu_seqlens,
                                        int32_t meta_type, int64_t max_seqlen, const ssu_slot_table *read,
                                        const ssu_slot_table *dst, void *workspace, uint64_t workspace_bytes,
                                        void *stream) {
    if (nseq < 0 || max_seqlen < 0) return fail(SSU_ERR_INVALID, "nseq and max_seqlen must not be negative");
    ssu::LinattnParams lp;
    ssu_status st = linattn_prepare(args, read, dst, &lp);
    if (st != SSU_OK) return st;
    if (!valid_itype(meta_type)) return fail(SSU_ERR_INVALID, "meta_type %d is not an ssu_itype", meta_type);
    if (args->io_dtype == SSU_F32) return fail(SSU_ERR_UNSUPPORTED, "the prefill takes fp16 or bf16 q, k, v and out");
    if (nseq == 0) return ok();
    if (!cu_seqlens) return fail(SSU_ERR_INVALID, "cu_seqlens must not be NULL");
    if (!aligned(cu_seqlens, itype_size(meta_type))) return fail(SSU_ERR_INVALID, "cu_seqlens must be aligned to its type");
    if (lp.rows > 0) {
        for (const void *q : {args->q, args->k, args->v, static_cast<const void *>(args->out)})
            if (!aligned16(q)) return fail(SSU_ERR_INVALID, "q, k, v and out must be 16-byte aligned");
        for (int i = 0; i < 2; ++i)
            if (lp.qs[i] % 8 || lp.ks[i] % 8 || lp.vs[i] % 8 || lp.os[i] % 8)
                return fail(SSU_ERR_INVALID, "the strides of q, k, v and out must be multiples of 8");
    }
    if (lp.rows >= kMaxGrid) return fail(SSU_ERR_INVALID, "more than 2^31-1 tokens");
    if (nseq > kMaxGrid / (4 * lp.H) || lp.rows / 128 > kMaxGrid / (4 * lp.H))
        return fail(SSU_ERR_INVALID, "too many sequences, tokens and heads for one call");
    const ssu::LinattnSplit split = ssu::linattn_split(lp.rows, nseq, lp.H, lp.P, lp.N, max_seqlen);
    if (split.bytes > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
        return fail(SSU_ERR_INVALID, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < split.bytes)
        return fail(SSU_ERR_INVALID, "workspace of %llu bytes is smaller than the %llu needed",
                    (unsigned long long)workspace_bytes, (unsigned long long)split.bytes);
    lp.nseq = nseq;
    lp.cu = cu_seqlens;
    lp.meta_is_i64 = meta_type == SSU_I64;
    if ((st = check_device(args->state)) != SSU_OK) return st;
    return launched(ssu::launch_linattn_prefill(lp, split, workspace, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_add_rmsnorm(const ssu_norm_args *a, void *stream) {
    if (a == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (!valid_dtype(a->dtype)) return fail(SSU_ERR_INVALID, "dtype %d is not an ssu_dtype", a->dtype);
    if (a->weight_dtype != a->dtype && a->weight_dtype != SSU_F32)
        return fail(SSU_ERR_INVALID, "weight has x's type or fp32");
    if (a->format != SSU_NORM_PLAIN && a->format != SSU_NORM_ROW && a->format != SSU_NORM_BLOCK)
        return fail(SSU_ERR_INVALID, "format %d is not an SSU_NORM_* value", a->format);
    if (a->rows < 0 || a->hidden < 1) return fail(SSU_ERR_INVALID, "rows must be >= 0 and hidden positive");
    if (a->hidden > ssu::kNormMaxHidden)
        return fail(SSU_ERR_UNSUPPORTED, "hidden %lld is not supported (up to %d)", (long long)a->hidden,
                    ssu::kNormMaxHidden);
    if (!(a->eps > 0.f)) return fail(SSU_ERR_INVALID, "eps must be positive");
    if (a->x_stride < 0 || a->residual_stride < 0 || a->residual_out_stride < 0 || a->y_stride < 0)
        return fail(SSU_ERR_INVALID, "a stride is negative");
    if (a->rows == 0) return ok();
    if ((a->residual == nullptr) != (a->residual_out == nullptr))
        return fail(SSU_ERR_INVALID, "residual and residual_out go together");
    if ((a->format == SSU_NORM_PLAIN) != (a->scales == nullptr))
        return fail(SSU_ERR_INVALID, "scales go with the E4M3 formats and only with them");
    if (!a->x || !a->weight || !a->y) return fail(SSU_ERR_INVALID, "x, weight and y must not be NULL");
    if (a->rows > kMaxGrid) return fail(SSU_ERR_INVALID, "more than 2^31-1 rows");
    for (const void *q : {a->x, a->residual, static_cast<const void *>(a->residual_out)})
        if (!aligned(q, dtype_size(a->dtype)))
            return fail(SSU_ERR_INVALID, "x, residual and residual_out must be aligned to their type");
    if (!aligned(a->weight, dtype_size(a->weight_dtype)) || !aligned(a->scales, 4) ||
        (a->format == SSU_NORM_PLAIN && !aligned(a->y, dtype_size(a->dtype))))
        return fail(SSU_ERR_INVALID, "weight, y and scales must be aligned to their type");
    if (a->y == a->x || a->y == a->residual || a->y == a->residual_out || (a->residual_out && a->residual_out == a->x))
        return fail(SSU_ERR_INVALID, "y must not alias x, residual or residual_out, nor residual_out x");
    ssu_status st = check_device(a->x, "x");
    if (st != SSU_OK) return st;
    ssu::NormParams p{};
    p.rows = a->rows;
    p.hidden = static_cast<int32_t>(a->hidden);
    p.dtype = a->dtype, p.weight_dtype = a->weight_dtype, p.quant = a->format;
    p.eps = a->eps;
    p.x = a->x, p.residual = a->residual, p.weight = a->weight;
    p.residual_out = a->residual_out, p.y = a->y, p.scales = a->scales;
    p.xs = a->x_stride, p.rs = a->residual_stride, p.ros = a->residual_out_stride, p.ys = a->y_stride;
    return launched(ssu::launch_norm(p, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_token_logprobs(const ssu_logprob_args *a, void *stream) {
    if (a == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (a->reserved0 != 0) return fail(SSU_ERR_INVALID, "reserved0 must be 0");
    if (!valid_dtype(a->dtype)) return fail(SSU_ERR_INVALID, "dtype %d is not an ssu_dtype", a->dtype);
    if (!valid_itype(a->token_type)) return fail(SSU_ERR_INVALID, "token_type %d is not an ssu_itype", a->token_type);
    if (a->rows < 0 || a->vocab < 1 || a->vocab > (1 << 30))
        return fail(SSU_ERR_INVALID, "rows must be >= 0 and vocab in [1, 2^30]");
    if (a->row_stride < 0) return fail(SSU_ERR_INVALID, "row_stride is negative");
    if (a->top_k < 0 || a->top_k > ssu::kMaxTopK || a->top_k > a->vocab)
        return fail(SSU_ERR_INVALID, "top_k %d: from 0 to %d and to vocab", a->top_k, ssu::kMaxTopK);
    if (a->rows == 0) return ok();
    if (!a->logits || !a->tokens || !a->logprobs || !a->entropy)
        return fail(SSU_ERR_INVALID, "logits, tokens, logprobs and entropy must not be NULL");
    if (a->top_k > 0 && (!a->top_ids || !a->top_logprobs))
        return fail(SSU_ERR_INVALID, "top_ids and top_logprobs must not be NULL");
    if (!aligned(a->logits, dtype_size(a->dtype))) return fail(SSU_ERR_INVALID, "logits must be aligned to their type");
    if (!aligned(a->tokens, itype_size(a->token_type)) || !aligned(a->top_ids, itype_size(a->token_type)))
        return fail(SSU_ERR_INVALID, "tokens and top_ids must be aligned to their type");
    for (const void *q : {static_cast<const void *>(a->logprobs), static_cast<const void *>(a->entropy),
                          static_cast<const void *>(a->top_logprobs), static_cast<const void *>(a->d_status)})
        if (!aligned(q, 4)) return fail(SSU_ERR_INVALID, "logprobs, entropy, top_logprobs and d_status must be 4-byte aligned");
    if (a->rows > kMaxGrid / 8) return fail(SSU_ERR_INVALID, "too many rows for one launch");
    ssu_status st = check_device(a->logits, "logits");
    if (st != SSU_OK) return st;
    ssu::LogprobParams p{};
    p.rows = a->rows, p.row_stride = a->row_stride;
    p.vocab = static_cast<int32_t>(a->vocab);
    p.dtype = a->dtype, p.top_k = a->top_k, p.tok_is_i64 = a->token_type == SSU_I64;
    p.logits = a->logits, p.tokens = a->tokens;
    p.logprob = a->logprobs, p.entropy = a->entropy;
    p.top_ids = a->top_ids, p.top_logprob = a->top_logprobs;
    p.status = a->d_status;
    return launched(ssu::launch_logprobs(p, static_cast<cudaStream_t>(stream)));
}

// Checks shared by the calls on a paged cache; fills `c`.
static ssu_status paged_prepare(const ssu_paged_args *a, ssu::PagedParams *c) {
    if (a == nullptr) return fail(SSU_ERR_INVALID, "args is NULL");
    if (a->reserved0 != 0) return fail(SSU_ERR_INVALID, "reserved0 must be 0");
    if (!valid_dtype(a->io_dtype)) return fail(SSU_ERR_INVALID, "io_dtype %d is not an ssu_dtype", a->io_dtype);
    if (a->io_dtype == SSU_F32) return fail(SSU_ERR_UNSUPPORTED, "a paged cache holds fp16 or bf16");
    if (!valid_itype(a->table_type)) return fail(SSU_ERR_INVALID, "table_type %d is not an ssu_itype", a->table_type);
    if (!valid_itype(a->meta_type)) return fail(SSU_ERR_INVALID, "meta_type %d is not an ssu_itype", a->meta_type);
    if (a->rows < 0 || a->nseq < 0) return fail(SSU_ERR_INVALID, "rows and nseq must not be negative");
    if (a->pages <= 0 || a->pages > kMaxGrid) return fail(SSU_ERR_INVALID, "pages must be positive and below 2^31");
    if (a->page_size <= 0) return fail(SSU_ERR_INVALID, "page_size must be positive");
    if (a->page_size % 8 != 0 || a->page_size > (1 << 20))
        return fail(SSU_ERR_UNSUPPORTED, "page_size %lld is not supported (multiples of 8 up to 2^20)", (long long)a->page_size);
    if (a->heads <= 0 || a->kv_heads <= 0 || a->heads % a->kv_heads != 0)
        return fail(SSU_ERR_INVALID, "heads (%lld) must be a positive multiple of kv_heads (%lld)", (long long)a->heads,
                    (long long)a->kv_heads);
    if (a->heads > 65535) return fail(SSU_ERR_INVALID, "more than 65535 heads");
    if (a->heads / a->kv_heads > ssu::kPagedMaxShare)
        return fail(SSU_ERR_UNSUPPORTED, "more than %d heads share a key/value head", ssu::kPagedMaxShare);
    if (a->dim < 8 || a->dim > ssu::kPagedMaxDim || a->dim % 8 != 0)
        return fail(SSU_ERR_UNSUPPORTED, "dim %lld is not supported (multiples of 8 from 8 to %d)", (long long)a->dim,
                    ssu::kPagedMaxDim);
    if (a->rows >= kMaxGrid || a->nseq >= kMaxGrid) return fail(SSU_ERR_INVALID, "more than 2^31-1 rows or sequences");
    if (a->rows + a->nseq > (kMaxGrid - (1 << 20)) / a->kv_heads)
        return fail(SSU_ERR_INVALID, "too many rows, sequences and heads for one call");
    if (a->cu_seqlens == nullptr && a->rows != a->nseq)
        return fail(SSU_ERR_INVALID, "without cu_seqlens every sequence has one row (rows %lld, nseq %lld)", (long long)a->rows,
                    (long long)a->nseq);
    if (a->table_width < 0 || a->table_stride < 0) return fail(SSU_ERR_INVALID, "table_width and table_stride must not be negative");
    if (!a->k_cache || !a->v_cache) return fail(SSU_ERR_INVALID, "k_cache and v_cache must not be NULL");
    if (a->k_cache == a->v_cache) return fail(SSU_ERR_INVALID, "k_cache and v_cache must not be the same");
    if (!aligned16(a->k_cache) || !aligned16(a->v_cache)) return fail(SSU_ERR_INVALID, "the caches must be 16-byte aligned");
    if (!aligned16(a->q) || !aligned16(a->out)) return fail(SSU_ERR_INVALID, "q and out must be 16-byte aligned");
    const int64_t extents[3] = {a->pages, a->page_size, a->kv_heads};
    for (int i = 0; i < 3; ++i)
        for (const int64_t s : {a->k_cache_stride[i], a->v_cache_stride[i]}) {
            if (extents[i] == 1) continue;
            if (s <= 0 || s % 8 != 0) return fail(SSU_ERR_INVALID, "the caches' strides must be positive multiples of 8");
            if (s >= (int64_t(1) << 39)) return fail(SSU_ERR_INVALID, "a stride of the caches is too large");
        }
    const int64_t across[2] = {a->rows, a->heads};
    for (int i = 0; i < 2; ++i)
        for (const int64_t s : {a->q ? a->q_stride[i] : 8, a->out ? a->out_stride[i] : 8})
            if (across[i] > 1 && (s <= 0 || s % 8 != 0 || s >= (int64_t(1) << 39)))
                return fail(SSU_ERR_INVALID, "the strides of q and out must be positive multiples of 8");
    if (!aligned(a->d_status, 4)) return fail(SSU_ERR_INVALID, "d_status must be 4-byte aligned");
    if (a->nseq > 0) {
        if (!a->kv_lens) return fail(SSU_ERR_INVALID, "kv_lens must not be NULL");
        if (a->table_width > 0 && !a->block_table) return fail(SSU_ERR_INVALID, "block_table must not be NULL");
        if (!aligned(a->kv_lens, itype_size(a->meta_type)) || !aligned(a->cu_seqlens, itype_size(a->meta_type)) ||
            !aligned(a->block_table, itype_size(a->table_type)))
            return fail(SSU_ERR_INVALID, "kv_lens, cu_seqlens and block_table must be aligned to their type");
    }
    std::memset(c, 0, sizeof *c);
    c->pages = a->pages, c->rows = a->rows, c->nseq = a->nseq;
    c->page = static_cast<int32_t>(a->page_size);
    c->H = static_cast<int32_t>(a->heads), c->G = static_cast<int32_t>(a->kv_heads), c->share = c->H / c->G;
    c->D = static_cast<int32_t>(a->dim);
    c->io_dtype = a->io_dtype;
    c->table_is_i64 = a->table_type == SSU_I64, c->meta_is_i64 = a->meta_type == SSU_I64;
    c->k_cache = a->k_cache, c->v_cache = a->v_cache;
    for (int i = 0; i < 3; ++i) c->ks[i] = a->k_cache_stride[i], c->vs[i] = a->v_cache_stride[i];
    c->table = a->block_table, c->table_stride = a->table_stride, c->table_width = a->table_width;
    c->kv_lens = a->kv_lens, c->cu = a->cu_seqlens;
    c->q = a->q, c->out = a->out;
    for (int i = 0; i < 2; ++i) c->qs[i] = a->q_stride[i], c->os[i] = a->out_stride[i];
    c->status = a->d_status;
    return SSU_OK;
}

ssu_status ssu_paged_append(const ssu_paged_args *args, const void *k, const int64_t *k_stride, const void *v,
                            const int64_t *v_stride, const float *inv_freq, int64_t rotary, int32_t interleaved,
                            void *stream) {
    ssu::AppendParams p{};
    ssu_status st = paged_prepare(args, &p.c);
    if (st != SSU_OK) return st;
    if (rotary < 0 || rotary > args->dim) return fail(SSU_ERR_INVALID, "rotary must be in [0, dim]");
    if (rotary % 16 != 0) return fail(SSU_ERR_UNSUPPORTED, "rotary %lld is not supported (multiples of 16)", (long long)rotary);
    if ((rotary > 0) != (inv_freq != nullptr)) return fail(SSU_ERR_INVALID, "inv_freq and a positive rotary go together");
    if (!aligned(inv_freq, 4)) return fail(SSU_ERR_INVALID, "inv_freq must be 4-byte aligned");
    if ((args->q == nullptr) != (args->out == nullptr)) return fail(SSU_ERR_INVALID, "q and out go together");
    if (args->out == args->q && args->q &&
        (args->q_stride[0] != args->out_stride[0] || args->q_stride[1] != args->out_stride[1]))
        return fail(SSU_ERR_INVALID, "q turned in place keeps its strides");
    if (args->rows == 0 || args->nseq == 0) return ok();
    if (!k || !v || !k_stride || !v_stride) return fail(SSU_ERR_INVALID, "k, v and their strides must not be NULL");
    if (!aligned16(k) || !aligned16(v)) return fail(SSU_ERR_INVALID, "k and v must be 16-byte aligned");
    for (int i = 0; i < 2; ++i) {
        if ((i == 0 ? args->rows : args->kv_heads) > 1 && (k_stride[i] < 0 || v_stride[i] < 0 || k_stride[i] % 8 || v_stride[i] % 8))
            return fail(SSU_ERR_INVALID, "the strides of k and v must be multiples of 8 and not negative");
        p.kstr[i] = k_stride[i], p.vstr[i] = v_stride[i];
    }
    for (const void *q : {k, v, args->q})
        if (q == args->k_cache || q == args->v_cache) return fail(SSU_ERR_INVALID, "k, v and q must not alias the caches");
    if (args->out && (args->out == k || args->out == v || args->out == args->k_cache || args->out == args->v_cache))
        return fail(SSU_ERR_INVALID, "out must not alias k, v or the caches");
    p.k = k, p.v = v;
    p.inv_freq = inv_freq;
    p.rotary = static_cast<int32_t>(rotary);
    p.interleaved = interleaved != 0;
    if ((st = check_device(args->k_cache, "k_cache")) != SSU_OK) return st;
    return launched(ssu::launch_paged_append(p, static_cast<cudaStream_t>(stream)));
}

// Checks of the attention's own arguments; fills `p` but for lse.
static ssu_status attend_prepare(const ssu_paged_args *args, float scale, int64_t window, int64_t max_seqlen,
                                 int64_t max_kv_len, ssu::AttendParams *p) {
    const ssu_status st = paged_prepare(args, &p->c);
    if (st != SSU_OK) return st;
    // (scores are taken in units of log2)
    if (!(scale > 0.f) || !(scale <= 2e38f)) return fail(SSU_ERR_INVALID, "scale must be positive and at most 2e38");
    if (window < 0) return fail(SSU_ERR_INVALID, "window must not be negative");
    if (max_seqlen < 0 || max_kv_len < 0) return fail(SSU_ERR_INVALID, "max_seqlen and max_kv_len must not be negative");
    p->scale = scale;
    // (a window longer than any sequence is none)
    p->window = window > ssu::kPagedMaxLen ? 0 : static_cast<int32_t>(window);
    p->lse = nullptr;
    return SSU_OK;
}

ssu_status ssu_paged_attention_workspace_size(const ssu_paged_args *args, int64_t max_seqlen, int64_t max_kv_len,
                                              uint64_t *bytes) {
    if (!bytes) return fail(SSU_ERR_INVALID, "bytes is NULL");
    ssu::AttendParams p{};
    const ssu_status st = attend_prepare(args, 1.f, 0, max_seqlen, max_kv_len, &p);
    if (st != SSU_OK) return st;
    *bytes = p.c.rows == 0 || p.c.nseq == 0 ? 0 : ssu::attend_plan(p, max_seqlen, max_kv_len).bytes;
    return ok();
}

ssu_status ssu_paged_attention(const ssu_paged_args *args, float scale, int64_t window, int64_t max_seqlen,
                               int64_t max_kv_len, float *lse, void *workspace, uint64_t workspace_bytes, void *stream) {
    ssu::AttendParams p{};
    ssu_status st = attend_prepare(args, scale, window, max_seqlen, max_kv_len, &p);
    if (st != SSU_OK) return st;
    if (p.c.rows == 0 || p.c.nseq == 0) return ok();
    if (!args->q || !args->out) return fail(SSU_ERR_INVALID, "q and out must not be NULL");
    if (args->out == args->q || args->out == args->k_cache || args->out == args->v_cache)
        return fail(SSU_ERR_INVALID, "out must not alias an input");
    if (!aligned(lse, 4)) return fail(SSU_ERR_INVALID, "lse must be 4-byte aligned");
    const ssu::AttendPlan plan = ssu::attend_plan(p, max_seqlen, max_kv_len);
    if (plan.bytes > 0 && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
        return fail(SSU_ERR_INVALID, "workspace must be a 256-byte aligned device pointer");
    if (workspace_bytes < plan.bytes)
        return fail(SSU_ERR_INVALID, "workspace of %llu bytes is smaller than the %llu needed",
                    (unsigned long long)workspace_bytes, (unsigned long long)plan.bytes);
    p.lse = lse;
    if ((st = check_device(args->k_cache, "k_cache")) != SSU_OK) return st;
    return launched(ssu::launch_paged_attention(p, plan, workspace, static_cast<cudaStream_t>(stream)));
}

ssu_status ssu_prewarm(int32_t state_dtype, int32_t io_dtype, int32_t dt_dtype, int64_t heads, int64_t dim,
                       int64_t dstate, int64_t groups, int32_t packed) {
    int lanes = 0;
    ssu_status st = check_shape(state_dtype, io_dtype, dt_dtype, heads, dim, dstate, groups, &lanes);
    if (st != SSU_OK) return st;
    cudaError_t e = packed ? ssu::prewarm_packed(state_dtype, lanes) : ssu::prewarm_onetoken(state_dtype, lanes);
    if (e != cudaSuccess) return fail(SSU_ERR_CUDA, "loading the kernel failed: %s", cudaGetErrorString(e));
    return ok();
}

const char *ssu_last_error(void) { return g_err; }

}  // extern "C"
