// zeroflat_api.cpp -- the extern "C" entry points of libzeroflat: argument
// validation, the FlatParameter layout (host integer arithmetic), the
// host-side scalars of the AdamW step, and dispatch to the gfx950 kernels.
// Nothing here allocates device memory or synchronizes.
#include <math.h>
#include <stdarg.h>
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <string>

#include "zeroflat.h"
#include "zf_launch.h"

namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return code;
}

int ok() {
    g_err.clear();
    return ZERO_OK;
}

int hip_fail(int e, const char* where) {
    return fail(ZERO_EHIP, "%s: HIP error %d (%s)", where, e, zf::hip_error_string(e));
}

bool valid_dtype(int32_t d) { return d == ZERO_F32 || d == ZERO_F16 || d == ZERO_BF16; }
int esize(int32_t d) { return d == ZERO_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

// the cache line the streaming reads are laid out on
constexpr uintptr_t kLineBytes = 128;

// the device address of the state's per-block partial-sum table (the state
// pointer is a device address: computed, never dereferenced, here)
double* state_partials(zero_step_state_t* st) {
    return st ? reinterpret_cast<double*>(reinterpret_cast<char*>(st) +
                                          offsetof(zero_step_state_t, partials))
              : nullptr;
}

// a*b, false on int64 overflow
bool mul_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_mul_overflow(a, b, out); }
bool add_ok(int64_t a, int64_t b, int64_t* out) { return !__builtin_add_overflow(a, b, out); }

}  // namespace

extern "C" {

const char* zero_last_error(void) { return g_err.c_str(); }

// ---------------------------------------------------------------------------
// FlatParameter layout ("PyTorch FSDP 源码级深度解析" §3.1 offsets; equal
// padded shards so that every rank's Reduce-Scatter output has one size,
// §3.3) and per-rank accounting ("DeepSpeed 与 FSDP", ZeRO-3 的数学总结).
int zero_flat_layout(const int64_t* numels, int32_t n_params, int32_t n_ranks, int64_t align,
                     int32_t param_bytes, int32_t grad_bytes, int32_t optim_bytes,
                     int32_t rank, zero_layout_t* out, zero_span_t* spans,
                     zero_segment_t* segs, int32_t segs_cap, int32_t* n_segs) {
    if (!out) return fail(ZERO_EINVAL, "zero_flat_layout: out is NULL");
    if (n_params < 0 || (n_params > 0 && !numels))
        return fail(ZERO_EINVAL, "zero_flat_layout: bad parameter list");
    if (n_ranks < 1) return fail(ZERO_EINVAL, "zero_flat_layout: n_ranks must be >= 1");
    if (align < 1) return fail(ZERO_EINVAL, "zero_flat_layout: align must be >= 1");
    if (rank < 0 || rank >= n_ranks) return fail(ZERO_EINVAL, "zero_flat_layout: rank out of range");
    if (param_bytes < 0 || grad_bytes < 0 || optim_bytes < 0)
        return fail(ZERO_EINVAL, "zero_flat_layout: negative byte counts");
    if (segs_cap < 0 || (segs_cap > 0 && !segs))
        return fail(ZERO_EINVAL, "zero_flat_layout: bad segment buffer");

    int64_t total = 0;
    for (int32_t j = 0; j < n_params; ++j) {
        if (numels[j] < 0) return fail(ZERO_EINVAL, "zero_flat_layout: numel[%d] < 0", j);
        if (!add_ok(total, numels[j], &total)) return fail(ZERO_ERANGE, "zero_flat_layout: total overflows");
    }
    // S = ceil(T / N) rounded up to a multiple of align
    int64_t shard = total / n_ranks + (total % n_ranks ? 1 : 0);
    const int64_t rem = shard % align;
    if (rem && !add_ok(shard, align - rem, &shard))
        return fail(ZERO_ERANGE, "zero_flat_layout: shard overflows");
    int64_t padded;
    if (!mul_ok(shard, n_ranks, &padded)) return fail(ZERO_ERANGE, "zero_flat_layout: padded overflows");

    zero_layout_t L;
    memset(&L, 0, sizeof L);
    L.total = total;
    L.shard = shard;
    L.padded = padded;
    L.pad = padded - total;
    L.n_ranks = n_ranks;
    L.align = align;
    const int64_t P = param_bytes, G = grad_bytes, K = optim_bytes;
    int64_t t0 = 0, t1 = 0, t2 = 0;
    bool good = mul_ok(P + G + K, total, &L.bytes_dp);
    good = good && mul_ok(P + G, total, &t0) && mul_ok(K, shard, &t1) && add_ok(t0, t1, &L.bytes_z1);
    good = good && mul_ok(P, total, &t0) && mul_ok(G + K, shard, &t1) && add_ok(t0, t1, &L.bytes_z2);
    good = good && mul_ok(P + G + K, shard, &t2);
    L.bytes_z3 = t2;
    if (!good) return fail(ZERO_ERANGE, "zero_flat_layout: byte accounting overflows");
    *out = L;

    // pieces of rank r's shard [r*S, (r+1)*S): parameters in order, then padding
    const int64_t lo_r = (int64_t)rank * shard, hi_r = lo_r + shard;
    int32_t count = 0;
    int64_t start = 0;
    for (int32_t j = 0; j <= n_params; ++j) {
        const int64_t s = j < n_params ? start : total;
        const int64_t e = j < n_params ? start + numels[j] : padded;
        if (spans && j < n_params) { spans[j].start = s; spans[j].end = e; }
        if (j < n_params) start = e;
        const int64_t lo = s > lo_r ? s : lo_r;
        const int64_t hi = e < hi_r ? e : hi_r;
        if (lo >= hi) continue;
        if (segs && count < segs_cap) {
            segs[count].param = j < n_params ? j : -1;
            segs[count].reserved = 0;
            segs[count].off_in_param = lo - s;
            segs[count].off_in_shard = lo - lo_r;
            segs[count].len = hi - lo;
        }
        ++count;
    }
    if (n_segs) *n_segs = count;
    if (segs && count > segs_cap)
        return fail(ZERO_ERANGE, "zero_flat_layout: %d segments do not fit in %d", count, segs_cap);
    return ok();
}

// ---------------------------------------------------------------------------
int zero_step_state_init(zero_step_state_t* st, float loss_scale, int32_t dynamic, int32_t window,
                         float min_scale) {
    if (!st) return fail(ZERO_EINVAL, "zero_step_state_init: state is NULL");
    if (!(min_scale >= 1.0f)) return fail(ZERO_EINVAL, "zero_step_state_init: min_scale must be >= 1");
    int ex;
    const float mant = frexpf(loss_scale, &ex);
    if (!(loss_scale >= min_scale) || mant != 0.5f || loss_scale > 1e38f)
        return fail(ZERO_EINVAL, "zero_step_state_init: loss_scale must be a power of two >= min_scale");
    if (dynamic && window < 1) return fail(ZERO_EINVAL, "zero_step_state_init: window must be >= 1");
    memset(st, 0, sizeof *st);
    st->loss_scale = loss_scale;
    st->min_scale = min_scale;
    st->dynamic = dynamic ? 1 : 0;
    st->window = window;
    st->beta1_pow = 1.0;
    st->beta2_pow = 1.0;
    return ok();
}

// ---------------------------------------------------------------------------
namespace {
// zero_grad_reduce_shard, zero_grad_accumulate_shard and
// zero_grad_reduce_shard_noalloc: the same reduce, the second adding into its
// output instead of overwriting it, the third keeping the statistics' partial
// sums in the library's device scratch instead of the state.
int reduce_entry(const char* fn, const void* const* grad_bufs, int32_t n_ranks, int32_t in_dtype,
                 int64_t elem_offset, int64_t shard_numel, int32_t op, float* red_out,
                 int accumulate, zero_step_state_t* d_state, void* stream, bool noalloc = false) {
    if (!grad_bufs) return fail(ZERO_EINVAL, "%s: grad_bufs is NULL", fn);
    if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS)
        return fail(ZERO_ERANGE, "%s: n_ranks %d not in [1, %d]", fn, n_ranks, ZERO_MAX_RANKS);
    if (!valid_dtype(in_dtype)) return fail(ZERO_EINVAL, "%s: bad in_dtype %d", fn, in_dtype);
    if (op != ZERO_SUM && op != ZERO_AVG) return fail(ZERO_EINVAL, "%s: bad op %d", fn, op);
    if (elem_offset < 0 || shard_numel < 0)
        return fail(ZERO_EINVAL, "%s: negative offset or size", fn);
    if (shard_numel == 0) return ok();  // nothing is read or written
    if (!red_out) return fail(ZERO_EINVAL, "%s: output shard is NULL", fn);
    if (!aligned(red_out, 4)) return fail(ZERO_EALIGN, "%s: output shard not 4-byte aligned", fn);
    if (d_state && !aligned(d_state, 8)) return fail(ZERO_EALIGN, "%s: state not 8-byte aligned", fn);
    const int es = esize(in_dtype);
    zf::ReduceLaunch a;
    memset(&a, 0, sizeof a);
    // vector path: each lane reads 4 consecutive inputs (8 B for 16-bit, 16 B
    // for fp32) and writes (and, accumulating, reads) 4 fp32 outputs (16 B).
    // Rank slices that all start at one offset within a quad keep it, wherever
    // they start ("PyTorch FSDP 源码级深度解析" §3.3: rank r's slice starts at
    // r*S, for any S): the elements up to the first slice's next 128-byte line
    // go element-wise, then the tiles read whole lines and their reduced quads
    // are shifted onto the aligned output.
    const uintptr_t quad = 4 * (uintptr_t)es;
    bool vec = aligned(red_out, 16);
    uintptr_t mis = 0, line_off = 0;
    for (int32_t k = 0; k < n_ranks; ++k) {
        if (!grad_bufs[k]) return fail(ZERO_EINVAL, "%s: grad_bufs[%d] is NULL", fn, k);
        if (!aligned(grad_bufs[k], es))
            return fail(ZERO_EALIGN, "%s: grad_bufs[%d] misaligned", fn, k);
        const char* p = static_cast<const char*>(grad_bufs[k]) + elem_offset * es;
        a.bufs[k] = p;
        const uintptr_t m = (uintptr_t)p % quad;
        if (k == 0) {
            mis = m;
            line_off = (uintptr_t)p % kLineBytes;
        }
        vec = vec && m == mis;
    }
    a.n_ranks = n_ranks;
    a.dtype = in_dtype;
    a.op = op;
    a.vec = vec ? 1 : 0;
    a.head = vec && line_off ? (int32_t)((kLineBytes - line_off) / es) : 0;
    a.n = shard_numel;
    a.red_out = red_out;
    a.accumulate = accumulate;
    a.st = d_state;
    a.partials = state_partials(d_state);
    const int e = noalloc ? zf::launch_reduce_noalloc(a, stream) : zf::launch_reduce_stats(a, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}
}  // namespace

int zero_grad_reduce_shard(const void* const* grad_bufs, int32_t n_ranks, int32_t in_dtype,
                           int64_t elem_offset, int64_t shard_numel, int32_t op,
                           float* red_out, zero_step_state_t* d_state, void* stream) {
    return reduce_entry("zero_grad_reduce_shard", grad_bufs, n_ranks, in_dtype, elem_offset,
                        shard_numel, op, red_out, 0, d_state, stream);
}

// The same reduce for callers that cannot allocate: the statistics' partial
// sums go to the library's per-device scratch, so d_state needs only the
// header of zero_step_state_t.
int zero_grad_reduce_shard_noalloc(const void* const* grad_bufs, int32_t n_ranks,
                                   int32_t in_dtype, int64_t elem_offset, int64_t shard_numel,
                                   int32_t op, float* red_out, zero_step_state_t* d_state,
                                   void* stream) {
    return reduce_entry("zero_grad_reduce_shard_noalloc", grad_bufs, n_ranks, in_dtype,
                        elem_offset, shard_numel, op, red_out, 0, d_state, stream, true);
}

// ---------------------------------------------------------------------------
// Gradient accumulation in the sharded state ("DeepSpeed 与 FSDP", 实践要点;
// 2kiu.com §5.3): acc += this micro-step's reduce.
int zero_grad_accumulate_shard(const void* const* grad_bufs, int32_t n_ranks, int32_t in_dtype,
                               int64_t elem_offset, int64_t shard_numel, int32_t op, float* acc,
                               zero_step_state_t* d_state, void* stream) {
    return reduce_entry("zero_grad_accumulate_shard", grad_bufs, n_ranks, in_dtype, elem_offset,
                        shard_numel, op, acc, 1, d_state, stream);
}

int zero_unscale_norm(const void* grad_shard, int32_t dtype, int64_t n, zero_step_state_t* d_state,
                      void* stream) {
    if (!d_state) return fail(ZERO_EINVAL, "zero_unscale_norm: NULL state");
    if (!valid_dtype(dtype)) return fail(ZERO_EINVAL, "zero_unscale_norm: bad dtype %d", dtype);
    if (n < 0) return fail(ZERO_EINVAL, "zero_unscale_norm: n < 0");
    if (n == 0) return ok();  // nothing is read
    if (!grad_shard) return fail(ZERO_EINVAL, "zero_unscale_norm: grad_shard is NULL");
    if (!aligned(grad_shard, esize(dtype))) return fail(ZERO_EALIGN, "zero_unscale_norm: grad misaligned");
    if (!aligned(d_state, 8)) return fail(ZERO_EALIGN, "zero_unscale_norm: state not 8-byte aligned");
    zf::ReduceLaunch a;
    memset(&a, 0, sizeof a);
    a.bufs[0] = grad_shard;
    a.n_ranks = 1;
    a.dtype = dtype;
    a.op = ZERO_SUM;
    // the vector path from the shard's first 128-byte line boundary on (the
    // head before it element-wise)
    const uintptr_t line_off = (uintptr_t)grad_shard % kLineBytes;
    a.vec = 1;
    a.head = line_off ? (int32_t)((kLineBytes - line_off) / esize(dtype)) : 0;
    a.n = n;
    a.red_out = nullptr;
    a.st = d_state;
    a.partials = state_partials(d_state);
    const int e = zf::launch_reduce_stats(a, stream);
    if (e) return hip_fail(e, "zero_unscale_norm");
    return ok();
}

// ---------------------------------------------------------------------------
int zero_adamw_shard_step(const void* grad_shard, int32_t grad_dtype, float* master,
                          float* exp_avg, float* exp_avg_sq, int64_t n, void* allgather_buf,
                          int32_t param_dtype, int64_t slot_offset, int8_t* q_buf,
                          float* q_scales, int64_t q_slot_offset, int64_t q_scale_offset,
                          int32_t q_block, const zero_adamw_hparams_t* hp, uint32_t flags,
                          zero_step_state_t* d_state, void* stream) {
    const char* fn = "zero_adamw_shard_step";
    if (!hp || !d_state) return fail(ZERO_EINVAL, "%s: NULL hp or state", fn);
    if (n < 0 || slot_offset < 0) return fail(ZERO_EINVAL, "%s: negative size or offset", fn);
    if (flags & ~ZERO_STEP_FINALIZE) return fail(ZERO_EINVAL, "%s: unknown flags 0x%x", fn, flags);
    if (!valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", fn, grad_dtype);
    if (param_dtype != ZERO_F16 && param_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: param_dtype must be fp16 or bf16", fn);
    if (n > 0 && (!grad_shard || !master || !exp_avg || !exp_avg_sq || !allgather_buf))
        return fail(ZERO_EINVAL, "%s: NULL tensor pointer", fn);
    if (!(hp->lr >= 0.0) || !(hp->eps > 0.0) || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) ||
        !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) || !(hp->weight_decay >= 0.0))
        return fail(ZERO_EINVAL, "%s: hyper-parameters out of range", fn);
    if (!aligned(d_state, 8)) return fail(ZERO_EALIGN, "%s: state not 8-byte aligned", fn);
    const bool quant = q_buf != nullptr;
    if (quant) {
        if (!q_scales) return fail(ZERO_EINVAL, "%s: q_scales is NULL", fn);
        if (q_block != 256) return fail(ZERO_EINVAL, "%s: q_block must be 256", fn);
        if (q_slot_offset < 0 || q_scale_offset < 0) return fail(ZERO_EINVAL, "%s: negative INT8 offset", fn);
        if (!aligned(q_scales, 4)) return fail(ZERO_EALIGN, "%s: q_scales misaligned", fn);
    }
    zf::AdamLaunch a;
    memset(&a, 0, sizeof a);
    const int ges = esize(grad_dtype);
    if (n > 0) {
        if (!aligned(grad_shard, ges) || !aligned(master, 4) || !aligned(exp_avg, 4) ||
            !aligned(exp_avg_sq, 4) || !aligned(allgather_buf, 2))
            return fail(ZERO_EALIGN, "%s: a tensor is not aligned to its element size", fn);
    }
    a.g = grad_shard;
    a.gdtype = grad_dtype;
    a.pdtype = param_dtype;
    a.p = master;
    a.m = exp_avg;
    a.v = exp_avg_sq;
    a.n = n;
    a.lp = static_cast<uint16_t*>(allgather_buf) + slot_offset;
    a.q = quant ? q_buf + q_slot_offset : nullptr;
    a.qs = quant ? q_scales + q_scale_offset : nullptr;
    // vector path: 16-byte fp32 quads and grad quads of 4*ges bytes; the slot
    // (8-byte quads) and the INT8 codes (4-byte quads) at any element offset:
    // rank r's slot starts at r*S ("PyTorch FSDP 源码级深度解析" §3.3), and
    // gfx950 carries out a vector store that is not aligned to its size (the
    // slot and codes are 3 of the update's 28-31 bytes per parameter)
    const bool vec = aligned(master, 16) && aligned(exp_avg, 16) && aligned(exp_avg_sq, 16) &&
                     aligned(grad_shard, 4 * ges);
    a.vec = vec ? 1 : 0;
    a.flags = flags;
    // step scalars formed in double and rounded once to fp32
    a.b1 = (float)hp->beta1;
    a.c1 = (float)(1.0 - hp->beta1);
    a.b2 = (float)hp->beta2;
    a.c2 = (float)(1.0 - hp->beta2);
    a.lr = (float)hp->lr;
    a.wdf = (float)(1.0 - hp->lr * hp->weight_decay);
    a.eps = (float)hp->eps;
    a.beta1 = hp->beta1;
    a.beta2 = hp->beta2;
    a.max_norm = hp->max_grad_norm;
    a.st = d_state;
    const int e = zf::launch_adamw(a, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

// ---------------------------------------------------------------------------
int zero_quant_allgather_slot(const void* slot, int32_t dtype, int64_t n, int32_t block,
                              int8_t* q_buf, int64_t q_slot_offset, float* q_scales,
                              int64_t q_scale_offset, void* stream) {
    const char* fn = "zero_quant_allgather_slot";
    if (dtype != ZERO_F16 && dtype != ZERO_BF16) return fail(ZERO_EINVAL, "%s: dtype must be fp16 or bf16", fn);
    if (block != 256) return fail(ZERO_EINVAL, "%s: block must be 256", fn);
    if (n < 0 || q_slot_offset < 0 || q_scale_offset < 0) return fail(ZERO_EINVAL, "%s: negative size", fn);
    if (n == 0) return ok();
    if (!slot || !q_buf || !q_scales) return fail(ZERO_EINVAL, "%s: NULL pointer", fn);
    if (!aligned(slot, 2) || !aligned(q_scales, 4)) return fail(ZERO_EALIGN, "%s: misaligned", fn);
    zf::QuantLaunch a;
    a.x = slot;
    a.dtype = dtype;
    a.n = n;
    a.q = q_buf + q_slot_offset;
    a.qs = q_scales + q_scale_offset;
    // 2: eight elements per lane (16-byte slot, 8-byte codes); 1: quad tiles
    a.vec = (aligned(slot, 16) && aligned(a.q, 8)) ? 2 : (aligned(slot, 8) && aligned(a.q, 4)) ? 1 : 0;
    const int e = zf::launch_quant(a, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

// ---------------------------------------------------------------------------
// Quantised gradient reduce ("DeepSpeed 与 FSDP", ZeRO++：量化通信压缩).
int zero_grad_reduce_shard_int8(const int8_t* const* q_bufs, const float* const* scale_bufs,
                                int32_t n_ranks, int64_t shard_numel, int32_t block, int32_t op,
                                float* red_out, zero_step_state_t* d_state, void* stream) {
    const char* fn = "zero_grad_reduce_shard_int8";
    if (!q_bufs || !scale_bufs) return fail(ZERO_EINVAL, "%s: NULL pointer table", fn);
    if (n_ranks < 1 || n_ranks > ZERO_MAX_RANKS / 2)
        return fail(ZERO_ERANGE, "%s: n_ranks %d not in [1, %d]", fn, n_ranks, ZERO_MAX_RANKS / 2);
    if (op != ZERO_SUM && op != ZERO_AVG) return fail(ZERO_EINVAL, "%s: bad op %d", fn, op);
    if (shard_numel < 0) return fail(ZERO_EINVAL, "%s: negative size", fn);
    if (block < 4 || block % 4 != 0) return fail(ZERO_EINVAL, "%s: block %d is not a positive multiple of 4", fn, block);
    if (shard_numel == 0) return ok();  // nothing is read or written
    if (!red_out) return fail(ZERO_EINVAL, "%s: red_out is NULL", fn);
    if (!aligned(red_out, 4)) return fail(ZERO_EALIGN, "%s: red_out not 4-byte aligned", fn);
    if (d_state && !aligned(d_state, 8)) return fail(ZERO_EALIGN, "%s: state not 8-byte aligned", fn);
    zf::ReduceLaunch a;
    memset(&a, 0, sizeof a);
    bool vec = aligned(red_out, 16);
    for (int32_t k = 0; k < n_ranks; ++k) {
        if (!q_bufs[k] || !scale_bufs[k]) return fail(ZERO_EINVAL, "%s: rank %d's payload is NULL", fn, k);
        if (!aligned(scale_bufs[k], 4)) return fail(ZERO_EALIGN, "%s: scale_bufs[%d] misaligned", fn, k);
        a.bufs[2 * k] = q_bufs[k];
        a.bufs[2 * k + 1] = scale_bufs[k];
        vec = vec && aligned(q_bufs[k], 4);
    }
    a.n_ranks = n_ranks;
    a.dtype = ZERO_F32;  // unused by the INT8 source
    a.op = op;
    a.vec = vec ? 1 : 0;
    a.n = shard_numel;
    a.red_out = red_out;
    a.block = block;
    a.block_shift = (block & (block - 1)) == 0 ? __builtin_ctz((unsigned)block) : -1;
    a.st = d_state;
    a.partials = state_partials(d_state);
    const int e = zf::launch_reduce_q8(a, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

// ---------------------------------------------------------------------------
// ZeRO-Offload ("DeepSpeed 与 FSDP", ZeRO-Offload; 2kiu.com §4.1, §5.1).
namespace {
int check_hp(const char* fn, const zero_adamw_hparams_t* hp) {
    if (!hp) return fail(ZERO_EINVAL, "%s: NULL hp", fn);
    if (!(hp->lr >= 0.0) || !(hp->eps > 0.0) || !(hp->beta1 >= 0.0 && hp->beta1 < 1.0) ||
        !(hp->beta2 >= 0.0 && hp->beta2 < 1.0) || !(hp->weight_decay >= 0.0))
        return fail(ZERO_EINVAL, "%s: hyper-parameters out of range", fn);
    return ZERO_OK;
}
}  // namespace

namespace {
// The gradient array and the 16-bit parameter array of the host step: either
// disjoint, or the very same array when the gradient is 16-bit too (in-place
// staging, each element's gradient read before its parameter is stored).
bool staging_ok(const void* g, int gsize, const void* lp, int64_t n) {
    if (g == lp) return gsize == 2;
    const uintptr_t g0 = reinterpret_cast<uintptr_t>(g), g1 = g0 + (uintptr_t)n * gsize;
    const uintptr_t l0 = reinterpret_cast<uintptr_t>(lp), l1 = l0 + (uintptr_t)n * 2;
    return g1 <= l0 || l1 <= g0;
}
}  // namespace

int zero_offload_adamw_host(const void* grad, int32_t grad_dtype, float* master, float* exp_avg,
                            float* exp_avg_sq, int64_t n, void* lp_out, int32_t param_dtype,
                            const zero_adamw_hparams_t* hp, const zero_step_state_t* host_state,
                            int32_t n_threads, int32_t* skipped) {
    const char* fn = "zero_offload_adamw_host";
    if (int e = check_hp(fn, hp)) return e;
    if (!host_state || !skipped) return fail(ZERO_EINVAL, "%s: NULL state or skipped", fn);
    if (!valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", fn, grad_dtype);
    if (param_dtype != ZERO_F16 && param_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: param_dtype must be fp16 or bf16", fn);
    if (n < 0 || n_threads < 0) return fail(ZERO_EINVAL, "%s: negative size or thread count", fn);
    if (n > 0 && (!grad || !master || !exp_avg || !exp_avg_sq || !lp_out))
        return fail(ZERO_EINVAL, "%s: NULL array", fn);
    if (n > 0 && (!aligned(grad, esize(grad_dtype)) || !aligned(master, 4) || !aligned(exp_avg, 4) ||
                  !aligned(exp_avg_sq, 4) || !aligned(lp_out, 2)))
        return fail(ZERO_EALIGN, "%s: an array is not aligned to its element size", fn);
    if (n > 0 && !staging_ok(grad, esize(grad_dtype), lp_out, n))
        return fail(ZERO_EINVAL, "%s: lp_out overlaps grad other than as the same 16-bit array", fn);
    int sk = 0;
    zf::offload_adam_host(grad, grad_dtype, master, exp_avg, exp_avg_sq, n, lp_out, param_dtype, *hp,
                          *host_state, n_threads, &sk);
    *skipped = sk;
    return ok();
}

int zero_offload_step(const void* d_grad, int32_t grad_dtype, int64_t n, float* h_master,
                      float* h_exp_avg, float* h_exp_avg_sq, void* h_grad_stage, void* h_lp_stage,
                      void* d_allgather, int32_t param_dtype, int64_t slot_offset,
                      const zero_adamw_hparams_t* hp, zero_step_state_t* d_state, int64_t chunk,
                      int32_t n_threads, void* stream) {
    const char* fn = "zero_offload_step";
    if (int e = check_hp(fn, hp)) return e;
    if (!d_state) return fail(ZERO_EINVAL, "%s: NULL state", fn);
    if (!aligned(d_state, 8)) return fail(ZERO_EALIGN, "%s: state not 8-byte aligned", fn);
    if (!valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", fn, grad_dtype);
    if (param_dtype != ZERO_F16 && param_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: param_dtype must be fp16 or bf16", fn);
    if (n < 0 || slot_offset < 0 || chunk < 0 || n_threads < 0)
        return fail(ZERO_EINVAL, "%s: negative size, offset, chunk or thread count", fn);
    if (n > 0 && (!d_grad || !h_master || !h_exp_avg || !h_exp_avg_sq || !h_grad_stage ||
                  !h_lp_stage || !d_allgather))
        return fail(ZERO_EINVAL, "%s: NULL pointer", fn);
    const int es = esize(grad_dtype);
    if (n > 0 && (!aligned(d_grad, es) || !aligned(h_grad_stage, es) || !aligned(h_master, 4) ||
                  !aligned(h_exp_avg, 4) || !aligned(h_exp_avg_sq, 4) || !aligned(h_lp_stage, 2) ||
                  !aligned(d_allgather, 2)))
        return fail(ZERO_EALIGN, "%s: a buffer is not aligned to its element size", fn);
    // chunks of one buffer are filled while other chunks of the other are
    // read: the two are disjoint, or one 16-bit buffer used in place
    if (n > 0 && !staging_ok(h_grad_stage, es, h_lp_stage, n))
        return fail(ZERO_EINVAL, "%s: the staging buffers overlap other than as one 16-bit buffer", fn);
    zf::OffloadLaunch a;
    memset(&a, 0, sizeof a);
    a.d_grad = d_grad;
    a.gdtype = grad_dtype;
    a.pdtype = param_dtype;
    a.n = n;
    a.h_p = h_master;
    a.h_m = h_exp_avg;
    a.h_v = h_exp_avg_sq;
    a.h_grad = h_grad_stage;
    a.h_lp = h_lp_stage;
    a.d_slot = n > 0 ? static_cast<uint16_t*>(d_allgather) + slot_offset : nullptr;
    a.chunk = chunk > 0 ? chunk : (int64_t)1 << 24;
    a.n_threads = n_threads;
    a.st = d_state;
    const int e = zf::offload_step(a, *hp, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

// ---------------------------------------------------------------------------
// INT8 All-Gather consumer ("DeepSpeed 与 FSDP", ZeRO++：量化通信压缩;
// 2kiu.com §4.2): the gathered slots back to the flat parameter.
int zero_dequant_allgather(const int8_t* q_buf, const float* q_scales, int32_t n_slots,
                           int64_t slot_numel, int32_t block, void* out, int32_t out_dtype,
                           void* stream) {
    const char* fn = "zero_dequant_allgather";
    if (!valid_dtype(out_dtype)) return fail(ZERO_EINVAL, "%s: bad out_dtype %d", fn, out_dtype);
    if (n_slots < 1 || n_slots > 65536) return fail(ZERO_ERANGE, "%s: n_slots %d not in [1, 65536]", fn, n_slots);
    if (slot_numel < 0) return fail(ZERO_EINVAL, "%s: negative slot_numel", fn);
    if (block < 4 || block % 4 != 0) return fail(ZERO_EINVAL, "%s: block %d is not a positive multiple of 4", fn, block);
    int64_t total = 0;
    if (!mul_ok(slot_numel, n_slots, &total) || !mul_ok(total, 4, &total))
        return fail(ZERO_ERANGE, "%s: n_slots * slot_numel overflows", fn);
    if (slot_numel == 0) return ok();
    if (!q_buf || !q_scales || !out) return fail(ZERO_EINVAL, "%s: NULL pointer", fn);
    const int es = esize(out_dtype);
    if (!aligned(q_scales, 4) || !aligned(out, es)) return fail(ZERO_EALIGN, "%s: misaligned", fn);
    zf::DequantLaunch a;
    memset(&a, 0, sizeof a);
    a.q = q_buf;
    a.qs = q_scales;
    a.out = out;
    a.out_dtype = out_dtype;
    a.block = block;
    a.n_slots = n_slots;
    a.slot_numel = slot_numel;
    // quad path: 4 codes (4 B) in, 4 outputs (8 B 16-bit, 16 B fp32) out per
    // lane; slot starts keep the alignment when slot_numel % 4 == 0
    a.vec = (slot_numel % 4 == 0 && aligned(q_buf, 4) && aligned(out, 4 * es)) ? 1 : 0;
    const int e = zf::launch_dequant(a, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

// ---------------------------------------------------------------------------
// The step over a list of tensors.
namespace {
int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b ? 1 : 0); }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// elements one block of the statistics pass reads: the smallest power of two
// from kMinSpan on that leaves at most kMaxSpans full spans
constexpr int64_t kMinSpan = 4096, kMaxSpans = 4096;
// bytes from the step's scalars to the copy of the state in a plan's image
constexpr int64_t kSnapshotAt = 256;

int check_plan(const char* fn, const zero_multi_plan_t* plan) {
    if (!plan) return fail(ZERO_EINVAL, "%s: NULL plan", fn);
    if (plan->n_tensors < 0 || plan->n_tensors > ZERO_MAX_TENSORS || plan->image_bytes <= 0 ||
        !valid_dtype(plan->grad_dtype) || plan->span < kMinSpan)
        return fail(ZERO_EINVAL, "%s: the plan is not one of zero_multi_plan_init", fn);
    return ZERO_OK;
}

zf::MultiNormLaunch norm_launch(const zero_multi_plan_t* plan, void* d_plan, int reset,
                                zero_step_state_t* st) {
    char* base = static_cast<char*>(d_plan);
    zf::MultiNormLaunch a;
    memset(&a, 0, sizeof a);
    a.entries = reinterpret_cast<const zf::MultiEntry*>(base);
    a.span_tensor = reinterpret_cast<const int32_t*>(base + plan->spans_off);
    a.tensor_sumsq = reinterpret_cast<double*>(base + plan->sumsq_off);
    a.partials = reinterpret_cast<double*>(base + plan->partials_off);
    a.snapshot = reinterpret_cast<zf::MultiState*>(base + plan->scalars_off + kSnapshotAt);
    a.span = plan->span;
    a.n_tensors = plan->n_tensors;
    a.n_spans = plan->n_spans;
    a.dtype = plan->grad_dtype;
    a.reset = reset;
    a.st = st;
    return a;
}
}  // namespace

int zero_multi_plan_init(const int64_t* numels, int32_t n_tensors, int32_t grad_dtype,
                         int32_t param_dtype, int32_t state_bits, zero_multi_plan_t* plan,
                         void* image, int64_t image_bytes) {
    const char* fn = "zero_multi_plan_init";
    if (!plan) return fail(ZERO_EINVAL, "%s: NULL plan", fn);
    if (n_tensors < 0 || (n_tensors > 0 && !numels))
        return fail(ZERO_EINVAL, "%s: bad tensor list", fn);
    if (n_tensors > ZERO_MAX_TENSORS)
        return fail(ZERO_ERANGE, "%s: more than %d tensors", fn, ZERO_MAX_TENSORS);
    if (!valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", fn, grad_dtype);
    if (param_dtype != ZERO_NONE && param_dtype != ZERO_F16 && param_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: param_dtype must be fp16, bf16 or none", fn);
    if (state_bits != 0 && state_bits != 8 && state_bits != 32)
        return fail(ZERO_EINVAL, "%s: state_bits must be 32, 8 or 0", fn);
    int64_t total = 0, rows = 0;
    for (int32_t k = 0; k < n_tensors; ++k) {
        if (numels[k] < 0) return fail(ZERO_EINVAL, "%s: numel[%d] < 0", fn, k);
        // 4-byte elements: byte counts stay far from int64's end
        if (numels[k] > ((int64_t)1 << 56) || !add_ok(total, numels[k], &total) ||
            total > ((int64_t)1 << 56))
            return fail(ZERO_ERANGE, "%s: total overflows", fn);
        rows += ceil_div(numels[k], ZERO_ROW);
    }
    int64_t span = kMinSpan;
    while (ceil_div(total, span) > kMaxSpans) span *= 2;
    int64_t spans = 0;
    for (int32_t k = 0; k < n_tensors; ++k) spans += ceil_div(numels[k], span);
    const int tile_rows = spans > zf::kMultiShortSpans ? zf::kMultiRowsLong
                          : rows > zf::kMultiTinyRows  ? zf::kMultiRowsShort
                                                       : zf::kMultiRowsTiny;
    const int64_t tile_elems = (int64_t)ZERO_ROW * tile_rows;
    int64_t tiles = 0;
    if (state_bits)
        for (int32_t k = 0; k < n_tensors; ++k) tiles += ceil_div(numels[k], tile_elems);
    // tile and row indices are 32-bit in the kernels
    if (tiles > 0x3fffffff || rows > 0x7fffffff)
        return fail(ZERO_ERANGE, "%s: the list is too long", fn);

    zero_multi_plan_t P;
    memset(&P, 0, sizeof P);
    P.total = total;
    P.rows = rows;
    P.n_tensors = n_tensors;
    P.grad_dtype = grad_dtype;
    P.param_dtype = param_dtype;
    P.state_bits = state_bits;
    P.n_tiles = (int32_t)tiles;
    P.n_spans = (int32_t)spans;
    P.span = span;
    int64_t off = 0;
    auto part = [&](int64_t bytes) { const int64_t at = off; off = round_up(off + bytes, 256); return at; };
    P.bind_bytes = (int64_t)n_tensors * (int64_t)sizeof(zf::MultiEntry);
    part(P.bind_bytes);
    P.tile_rows = tile_rows;
    static_assert(sizeof(zf::MultiScalars) <= kSnapshotAt, "the scalars precede the snapshot");
    P.scalars_off = part(kSnapshotAt + (int64_t)sizeof(zf::MultiState));
    P.tiles_off = part(tiles * 4);
    P.spans_off = part(spans * 4);
    P.sumsq_off = part((int64_t)n_tensors * 8);
    P.partials_off = part(spans * 8);
    P.image_bytes = off;
    if (image) {
        if (!aligned(image, 8)) return fail(ZERO_EALIGN, "%s: image not 8-byte aligned", fn);
        if (image_bytes < P.image_bytes)
            return fail(ZERO_ERANGE, "%s: image holds %lld of %lld bytes", fn, (long long)image_bytes,
                        (long long)P.image_bytes);
        char* base = static_cast<char*>(image);
        memset(base, 0, (size_t)P.image_bytes);
        auto* e = reinterpret_cast<zf::MultiEntry*>(base);
        auto* tile_tensor = reinterpret_cast<int32_t*>(base + P.tiles_off);
        auto* span_tensor = reinterpret_cast<int32_t*>(base + P.spans_off);
        int64_t row = 0, tile = 0, sp = 0;
        for (int32_t k = 0; k < n_tensors; ++k) {
            const int64_t r = ceil_div(numels[k], ZERO_ROW);
            const int64_t nt = state_bits ? ceil_div(numels[k], tile_elems) : 0;
            const int64_t ns = ceil_div(numels[k], span);
            e[k].numel = numels[k];
            e[k].row0 = row;
            e[k].tile0 = (int32_t)tile;
            e[k].span0 = (int32_t)sp;
            e[k].n_spans = (int32_t)ns;
            e[k].lr_mult = 1.0;
            e[k].decay_mult = 1.0;
            for (int64_t i = 0; i < nt; ++i) tile_tensor[tile + i] = k;
            for (int64_t i = 0; i < ns; ++i) span_tensor[sp + i] = k;
            row += r;
            tile += nt;
            sp += ns;
        }
    }
    *plan = P;
    return ok();
}

int zero_multi_bind(const zero_multi_plan_t* plan, const void* const* grads, void* const* params,
                    const double* lr_mult, const double* decay_mult, void* image) {
    const char* fn = "zero_multi_bind";
    if (int e = check_plan(fn, plan)) return e;
    if (!image && plan->n_tensors > 0) return fail(ZERO_EINVAL, "%s: NULL image", fn);
    if (!aligned(image, 8)) return fail(ZERO_EALIGN, "%s: image not 8-byte aligned", fn);
    const bool copy = plan->param_dtype != ZERO_NONE;
    const int32_t n = plan->n_tensors;
    if (n > 0 && (!grads || (copy && !params)))
        return fail(ZERO_EINVAL, "%s: NULL pointer table", fn);
    if (!copy && params) return fail(ZERO_EINVAL, "%s: the plan has no param_dtype", fn);
    auto* e = static_cast<zf::MultiEntry*>(image);
    const int es = esize(plan->grad_dtype);
    for (int32_t k = 0; k < n; ++k) {   // nothing is written on error
        if (e[k].numel > 0 && (!grads[k] || (copy && !params[k])))
            return fail(ZERO_EINVAL, "%s: tensor %d is NULL", fn, k);
        if (e[k].numel > 0 && (!aligned(grads[k], es) || (copy && !aligned(params[k], 2))))
            return fail(ZERO_EALIGN, "%s: tensor %d is not aligned to its element size", fn, k);
        if ((lr_mult && !(lr_mult[k] >= 0.0 && isfinite(lr_mult[k]))) ||
            (decay_mult && !(decay_mult[k] >= 0.0 && isfinite(decay_mult[k]))))
            return fail(ZERO_EINVAL, "%s: factors of tensor %d out of range", fn, k);
    }
    for (int32_t k = 0; k < n; ++k) {
        e[k].grad = grads[k];
        e[k].param = copy ? params[k] : nullptr;
        e[k].lr_mult = lr_mult ? lr_mult[k] : 1.0;
        e[k].decay_mult = decay_mult ? decay_mult[k] : 1.0;
    }
    return ok();
}

int zero_multi_unscale_norm(const zero_multi_plan_t* plan, void* d_plan, uint32_t flags,
                            zero_step_state_t* d_state, void* stream) {
    const char* fn = "zero_multi_unscale_norm";
    if (int e = check_plan(fn, plan)) return e;
    if (!d_plan || !d_state) return fail(ZERO_EINVAL, "%s: NULL plan buffer or state", fn);
    if (!aligned(d_plan, 256)) return fail(ZERO_EALIGN, "%s: plan buffer not 256-byte aligned", fn);
    if (!aligned(d_state, 8)) return fail(ZERO_EALIGN, "%s: state not 8-byte aligned", fn);
    if (flags & ~ZERO_MULTI_RESET) return fail(ZERO_EINVAL, "%s: unknown flags 0x%x", fn, flags);
    zf::MultiNormLaunch a = norm_launch(plan, d_plan, flags & ZERO_MULTI_RESET ? 1 : 0, d_state);
    a.snapshot = nullptr;
    const int e = zf::launch_multi_norm(a, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

int zero_multi_adamw_step(const zero_multi_plan_t* plan, void* d_plan, float* master,
                          void* exp_avg, void* exp_avg_sq, float* m_scale, float* v_scale,
                          const zero_adamw_hparams_t* hp, uint32_t seed, uint32_t flags,
                          zero_step_state_t* d_state, void* stream) {
    const char* fn = "zero_multi_adamw_step";
    if (int e = check_plan(fn, plan)) return e;
    if (int e = check_hp(fn, hp)) return e;
    if (!d_plan || !d_state) return fail(ZERO_EINVAL, "%s: NULL plan buffer or state", fn);
    if (flags & ~(ZERO_STEP_FINALIZE | ZERO_MULTI_STATISTICS))
        return fail(ZERO_EINVAL, "%s: unknown flags 0x%x", fn, flags);
    if (!aligned(d_plan, 256)) return fail(ZERO_EALIGN, "%s: plan buffer not 256-byte aligned", fn);
    if (!aligned(d_state, 8)) return fail(ZERO_EALIGN, "%s: state not 8-byte aligned", fn);
    if (plan->state_bits != 8 && plan->state_bits != 32)
        return fail(ZERO_EINVAL, "%s: the plan only serves the statistics", fn);
    const bool q8 = plan->state_bits == 8;
    // the 8-bit form's reciprocal of the denominator needs a normal number
    if (q8 && (float)hp->eps < 1.17549435e-38f)
        return fail(ZERO_EINVAL, "%s: 8-bit states need eps >= 2^-126", fn);
    if (plan->rows > 0) {
        if (!master || !exp_avg || !exp_avg_sq || (q8 && (!m_scale || !v_scale)))
            return fail(ZERO_EINVAL, "%s: NULL state arena", fn);
        const uintptr_t al = q8 ? 4 : 16;
        if (!aligned(master, 16) || !aligned(exp_avg, al) || !aligned(exp_avg_sq, al) ||
            (q8 && (!aligned(m_scale, 4) || !aligned(v_scale, 4))))
            return fail(ZERO_EALIGN, "%s: a state arena is misaligned", fn);
    }
    char* base = static_cast<char*>(d_plan);
    zf::MultiAdamLaunch a;
    memset(&a, 0, sizeof a);
    a.entries = reinterpret_cast<const zf::MultiEntry*>(base);
    a.tile_tensor = reinterpret_cast<const int32_t*>(base + plan->tiles_off);
    a.p = master;
    a.m = exp_avg;
    a.v = exp_avg_sq;
    a.ms = m_scale;
    a.vs = v_scale;
    a.n_tiles = plan->n_tiles;
    a.tile_rows = plan->tile_rows;
    a.gdtype = plan->grad_dtype;
    a.pdtype = plan->param_dtype;
    a.bits = plan->state_bits;
    a.b1 = (float)hp->beta1;
    a.c1 = (float)(1.0 - hp->beta1);
    a.b2 = (float)hp->beta2;
    a.c2 = (float)(1.0 - hp->beta2);
    a.eps = (float)hp->eps;
    zf::MultiStep step;
    memset(&step, 0, sizeof step);
    step.scalars = reinterpret_cast<zf::MultiScalars*>(base + plan->scalars_off);
    step.st = d_state;
    step.lr = hp->lr;
    step.wd = hp->weight_decay;
    step.beta1 = hp->beta1;
    step.beta2 = hp->beta2;
    step.max_norm = hp->max_grad_norm;
    step.seed = seed;
    step.advance = flags & ZERO_STEP_FINALIZE ? 1 : 0;
    a.scalars = step.scalars;
    const bool stats = (flags & ZERO_MULTI_STATISTICS) != 0;
    const zf::MultiNormLaunch norm = norm_launch(plan, d_plan, 0, d_state);
    const int e = zf::launch_multi_step(a, stats ? &norm : nullptr, step, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

int zero_multi_adamw_step_args(const zero_multi_step_args_t* args, void* stream) {
    if (!args) return fail(ZERO_EINVAL, "zero_multi_adamw_step_args: NULL args");
    return zero_multi_adamw_step(args->plan, args->d_plan, args->master, args->exp_avg,
                                 args->exp_avg_sq, args->m_scale, args->v_scale, &args->hp,
                                 args->seed, args->flags, args->d_state, stream);
}

// ---------------------------------------------------------------------------
// 10. Embedding rows and their gradient.
namespace {
constexpr int64_t kEmbedMaxTokens = (int64_t)1 << 28, kEmbedMaxVocab = (int64_t)1 << 25;
constexpr int64_t kMaxCols = (int64_t)1 << 24;

int check_tokens(const char* fn, const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t first,
                 int64_t vocab, int64_t dim) {
    if (token_bytes != 4 && token_bytes != 8)
        return fail(ZERO_EINVAL, "%s: token_bytes must be 4 or 8", fn);
    if (n_tokens < 0 || first < 0 || vocab < 0 || dim < 0)
        return fail(ZERO_EINVAL, "%s: negative size or first token", fn);
    if (n_tokens > kEmbedMaxTokens || vocab > kEmbedMaxVocab || dim > kMaxCols)
        return fail(ZERO_ERANGE, "%s: more than 2^28 tokens, 2^25 rows or 2^24 columns", fn);
    if (n_tokens > 0 && !tokens) return fail(ZERO_EINVAL, "%s: NULL tokens", fn);
    if (!aligned(tokens, token_bytes)) return fail(ZERO_EALIGN, "%s: tokens not aligned to their size", fn);
    return ZERO_OK;
}

// the table's own arguments are checked by the caller
int embed_lookup(const char* fn, zf::EmbedLookupLaunch& l, const void* tokens, int32_t token_bytes,
                 int64_t n_tokens, int64_t first, int64_t vocab, int64_t dim, float scale, void* out,
                 int32_t out_dtype, int64_t out_ld, void* stream) {
    if (!valid_dtype(out_dtype)) return fail(ZERO_EINVAL, "%s: bad out_dtype %d", fn, out_dtype);
    if (n_tokens > 1 && out_ld < dim) return fail(ZERO_EINVAL, "%s: out_ld is less than dim", fn);
    int64_t end;
    if (n_tokens > 1 && !mul_ok(n_tokens - 1, out_ld, &end))
        return fail(ZERO_ERANGE, "%s: the output's size overflows", fn);
    if (n_tokens == 0 || dim == 0) return ok();
    if (!out) return fail(ZERO_EINVAL, "%s: NULL out", fn);
    if (!aligned(out, esize(out_dtype))) return fail(ZERO_EALIGN, "%s: out not aligned to its element size", fn);
    l.args.tokens = tokens;
    l.args.wide = token_bytes == 8;
    l.args.out = out;
    l.args.out_ld = out_ld;
    l.args.first = first;
    l.args.vocab = vocab;
    l.args.scale = scale;
    l.n_tokens = n_tokens;
    l.dim = dim;
    l.out_dtype = out_dtype;
    const int e = zf::launch_embed_lookup(l, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}
}  // namespace

int zero_embed_lookup(const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t first,
                      const void* table, int32_t table_dtype, int64_t vocab, int64_t dim, float scale,
                      void* out, int32_t out_dtype, int64_t out_ld, void* stream) {
    const char* fn = "zero_embed_lookup";
    if (int e = check_tokens(fn, tokens, token_bytes, n_tokens, first, vocab, dim)) return e;
    if (!valid_dtype(table_dtype)) return fail(ZERO_EINVAL, "%s: bad table_dtype %d", fn, table_dtype);
    if (n_tokens > 0 && vocab > 0 && dim > 0 && !table) return fail(ZERO_EINVAL, "%s: NULL table", fn);
    if (!aligned(table, esize(table_dtype)))
        return fail(ZERO_EALIGN, "%s: table not aligned to its element size", fn);
    zf::EmbedLookupLaunch l;
    memset(&l, 0, sizeof l);
    l.args.table = table;
    l.table_dtype = table_dtype;
    return embed_lookup(fn, l, tokens, token_bytes, n_tokens, first, vocab, dim, scale, out, out_dtype, out_ld,
                        stream);
}

int zero_embed_lookup_int8(const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t first,
                           const int8_t* q_buf, const float* q_scales, int32_t n_slots,
                           int64_t slot_numel, int32_t block, int64_t elem_offset, int64_t vocab,
                           int64_t dim, float scale, void* out, int32_t out_dtype, int64_t out_ld,
                           void* stream) {
    const char* fn = "zero_embed_lookup_int8";
    if (int e = check_tokens(fn, tokens, token_bytes, n_tokens, first, vocab, dim)) return e;
    if (block != 256) return fail(ZERO_EINVAL, "%s: block must be 256", fn);
    if (n_slots < 1 || n_slots > 65536) return fail(ZERO_ERANGE, "%s: n_slots out of range", fn);
    if (slot_numel < 0 || elem_offset < 0) return fail(ZERO_EINVAL, "%s: negative slot size or offset", fn);
    int64_t held, need;
    if (!mul_ok(slot_numel, n_slots, &held) || !add_ok(vocab * dim, elem_offset, &need))
        return fail(ZERO_ERANGE, "%s: the payload's size overflows", fn);
    if (need > held) return fail(ZERO_EINVAL, "%s: the table exceeds the payload's slots", fn);
    if (n_tokens > 0 && vocab > 0 && dim > 0 && (!q_buf || !q_scales))
        return fail(ZERO_EINVAL, "%s: NULL payload", fn);
    if (!aligned(q_scales, 4)) return fail(ZERO_EALIGN, "%s: q_scales not 4-byte aligned", fn);
    zf::EmbedLookupLaunch l;
    memset(&l, 0, sizeof l);
    l.args.table = q_buf;
    l.args.scales = q_scales;
    l.args.elem_offset = elem_offset;
    l.args.slot_numel = slot_numel > 0 ? slot_numel : 1;
    l.args.slot_blocks = slot_numel / block + (slot_numel % block ? 1 : 0);
    l.table_dtype = zf::kEmbedInt8;
    return embed_lookup(fn, l, tokens, token_bytes, n_tokens, first, vocab, dim, scale, out, out_dtype, out_ld,
                        stream);
}

int zero_embed_grad_workspace(int64_t n_tokens, int64_t vocab, int64_t dim, int64_t* bytes) {
    const char* fn = "zero_embed_grad_workspace";
    if (!bytes) return fail(ZERO_EINVAL, "%s: NULL bytes", fn);
    if (int e = check_tokens(fn, &fn, 8, n_tokens, 0, vocab, dim)) return e;
    *bytes = zf::embed_workspace(n_tokens, vocab, dim).bytes;
    return ok();
}

int zero_embed_grad(const void* tokens, int32_t token_bytes, int64_t n_tokens, int64_t first,
                    const int64_t* padding, const void* dy, int32_t dy_dtype, int64_t dy_ld, float scale,
                    void* grad, int32_t grad_dtype, int64_t vocab, int64_t dim, uint32_t flags,
                    void* workspace, int64_t workspace_bytes, void* stream) {
    const char* fn = "zero_embed_grad";
    if (int e = check_tokens(fn, tokens, token_bytes, n_tokens, first, vocab, dim)) return e;
    if (!valid_dtype(dy_dtype) || !valid_dtype(grad_dtype))
        return fail(ZERO_EINVAL, "%s: bad dy_dtype %d or grad_dtype %d", fn, dy_dtype, grad_dtype);
    if (flags & ~ZERO_ACCUMULATE) return fail(ZERO_EINVAL, "%s: unknown flags", fn);
    if (dy_ld < 0) return fail(ZERO_EINVAL, "%s: negative dy_ld", fn);
    int64_t end;
    if (!mul_ok(n_tokens, dy_ld, &end)) return fail(ZERO_ERANGE, "%s: dy's size overflows", fn);
    const bool accumulate = flags & ZERO_ACCUMULATE;
    if (vocab == 0 || dim == 0 || (n_tokens == 0 && accumulate)) return ok();
    if (!grad || (n_tokens > 0 && !dy)) return fail(ZERO_EINVAL, "%s: NULL dy or grad", fn);
    if (!aligned(dy, esize(dy_dtype)) || !aligned(grad, esize(grad_dtype)))
        return fail(ZERO_EALIGN, "%s: dy or grad not aligned to its element size", fn);
    const zf::EmbedWorkspace w = zf::embed_workspace(n_tokens, vocab, dim);
    if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes))
        return fail(ZERO_EINVAL, "%s: the workspace needs %lld bytes", fn, (long long)w.bytes);
    if (w.bytes > 0 && !aligned(workspace, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", fn);
    // (a row distance of 0 asks for more sums than dy has memory)
    if (w.tiles * ((dim + 511) / 512) + vocab / 4 >= (int64_t)1 << 24)
        return fail(ZERO_ERANGE, "%s: more than 2^24 tiles of sums", fn);
    zf::EmbedGradLaunch l;
    memset(&l, 0, sizeof l);
    l.sort.tokens = tokens;
    l.sort.n_tokens = n_tokens;
    l.sort.first = first;
    l.sort.padding = padding ? *padding : 0;
    l.sort.has_padding = padding != nullptr;
    l.sort.vocab = vocab;
    l.sort.wide = token_bytes == 8;
    l.sum.dy = dy;
    l.sum.grad = grad;
    l.sum.dim = dim;
    l.sum.dy_ld = dy_ld;
    l.sum.accumulate = accumulate;
    l.sum.scale = scale;
    l.workspace = workspace;
    l.dy_dtype = dy_dtype;
    l.grad_dtype = grad_dtype;
    const int e = zf::launch_embed_grad(l, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

// ---------------------------------------------------------------------------
// 11. Activations kept in 8 bits.
namespace {
int check_matrix(const char* fn, const char* name, const void* p, int32_t dtype, int64_t rows, int64_t cols,
                 int64_t ld, bool written) {
    if (!p) return fail(ZERO_EINVAL, "%s: NULL %s", fn, name);
    if (!aligned(p, esize(dtype))) return fail(ZERO_EALIGN, "%s: %s not aligned to its element size", fn, name);
    int64_t end;
    if (ld < 0 || (written && rows > 1 && ld < cols))
        return fail(ZERO_EINVAL, "%s: bad row distance of %s", fn, name);
    if (!mul_ok(rows, ld, &end) || end > INT64_MAX / 8) return fail(ZERO_ERANGE, "%s: %s is too large", fn, name);
    return ZERO_OK;
}
int check_saved(const char* fn, const char* name, const int8_t* codes, const uint8_t* exponents) {
    if (!codes || !exponents) return fail(ZERO_EINVAL, "%s: NULL checkpoint (%s)", fn, name);
    if (!aligned(codes, 16)) return fail(ZERO_EALIGN, "%s: codes of %s not 16-byte aligned", fn, name);
    return ZERO_OK;
}
// 0: go on; 1: nothing to do; negative: an error
int check_act(const char* fn, int32_t dtype, int64_t rows, int64_t cols) {
    if (!valid_dtype(dtype)) return fail(ZERO_EINVAL, "%s: bad dtype %d", fn, dtype);
    if (rows < 0 || cols < 0) return fail(ZERO_EINVAL, "%s: negative size", fn);
    if (cols > kMaxCols || rows > (int64_t)1 << 40) return fail(ZERO_ERANGE, "%s: more than 2^40 rows or 2^24 columns", fn);
    return rows == 0 || cols == 0 ? 1 : 0;
}
zf::ActLaunch act_launch(int32_t kind, int32_t dtype, int64_t rows, int64_t cols) {
    zf::ActLaunch a;
    memset(&a, 0, sizeof a);
    a.rows = rows;
    a.cols = cols;
    a.dtype = dtype;
    a.kind = kind;
    a.least = dtype == ZERO_F16 ? 109 : 7;
    return a;
}
int run_act(const char* fn, const zf::ActLaunch& a, int backward, void* stream) {
    const int e = zf::launch_act(a, backward, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}
bool valid_kind(int32_t k) { return k == ZERO_GELU || k == ZERO_GELU_TANH || k == ZERO_SILU; }
}  // namespace

int zero_act_save8(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t x_ld, int8_t* codes,
                   uint8_t* exponents, void* stream) {
    const char* fn = "zero_act_save8";
    if (int e = check_act(fn, dtype, rows, cols)) return e < 0 ? e : ok();
    if (int e = check_matrix(fn, "x", x, dtype, rows, cols, x_ld, false)) return e;
    if (int e = check_saved(fn, "x", codes, exponents)) return e;
    zf::ActLaunch a = act_launch(-1, dtype, rows, cols);
    a.x = x;
    a.x_ld = x_ld;
    a.codes = codes;
    a.exponents = exponents;
    return run_act(fn, a, 0, stream);
}

int zero_act_restore8(const int8_t* codes, const uint8_t* exponents, int64_t rows, int64_t cols, void* out,
                      int32_t dtype, int64_t out_ld, void* stream) {
    const char* fn = "zero_act_restore8";
    if (int e = check_act(fn, dtype, rows, cols)) return e < 0 ? e : ok();
    if (int e = check_matrix(fn, "out", out, dtype, rows, cols, out_ld, true)) return e;
    if (int e = check_saved(fn, "x", codes, exponents)) return e;
    zf::ActLaunch a = act_launch(-1, dtype, rows, cols);
    a.y = out;
    a.y_ld = out_ld;
    a.codes = const_cast<int8_t*>(codes);
    a.exponents = const_cast<uint8_t*>(exponents);
    return run_act(fn, a, 1, stream);
}

int zero_act_forward8(int32_t kind, const void* x, int64_t x_ld, const void* up, int64_t up_ld, int32_t dtype,
                      int64_t rows, int64_t cols, void* y, int64_t y_ld, int8_t* codes, uint8_t* exponents,
                      int8_t* up_codes, uint8_t* up_exponents, void* stream) {
    const char* fn = "zero_act_forward8";
    if (!valid_kind(kind)) return fail(ZERO_EINVAL, "%s: bad kind %d", fn, kind);
    if (int e = check_act(fn, dtype, rows, cols)) return e < 0 ? e : ok();
    if (int e = check_matrix(fn, "x", x, dtype, rows, cols, x_ld, false)) return e;
    if (int e = check_matrix(fn, "y", y, dtype, rows, cols, y_ld, true)) return e;
    if (int e = check_saved(fn, "x", codes, exponents)) return e;
    zf::ActLaunch a = act_launch(kind, dtype, rows, cols);
    a.x = x;
    a.x_ld = x_ld;
    a.y = y;
    a.y_ld = y_ld;
    a.codes = codes;
    a.exponents = exponents;
    if (up) {
        if (int e = check_matrix(fn, "up", up, dtype, rows, cols, up_ld, false)) return e;
        if (int e = check_saved(fn, "up", up_codes, up_exponents)) return e;
        a.up = up;
        a.up_ld = up_ld;
        a.up_codes = up_codes;
        a.up_exponents = up_exponents;
    } else if (up_codes || up_exponents) {
        return fail(ZERO_EINVAL, "%s: a checkpoint of up without up", fn);
    }
    return run_act(fn, a, 0, stream);
}

int zero_act_backward8(int32_t kind, const void* dy, int64_t dy_ld, int32_t dtype, int64_t rows, int64_t cols,
                       const int8_t* codes, const uint8_t* exponents, const int8_t* up_codes,
                       const uint8_t* up_exponents, void* dx, int64_t dx_ld, void* dup, int64_t dup_ld,
                       int8_t* again_codes, uint8_t* again_exponents, void* stream) {
    const char* fn = "zero_act_backward8";
    if (!valid_kind(kind)) return fail(ZERO_EINVAL, "%s: bad kind %d", fn, kind);
    if (int e = check_act(fn, dtype, rows, cols)) return e < 0 ? e : ok();
    if (int e = check_matrix(fn, "dy", dy, dtype, rows, cols, dy_ld, false)) return e;
    if (int e = check_matrix(fn, "dx", dx, dtype, rows, cols, dx_ld, true)) return e;
    if (int e = check_saved(fn, "x", codes, exponents)) return e;
    zf::ActLaunch a = act_launch(kind, dtype, rows, cols);
    a.x = dy;
    a.x_ld = dy_ld;
    a.y = dx;
    a.y_ld = dx_ld;
    a.codes = const_cast<int8_t*>(codes);
    a.exponents = const_cast<uint8_t*>(exponents);
    if (up_codes || up_exponents) {
        if (int e = check_saved(fn, "up", up_codes, up_exponents)) return e;
        if (int e = check_matrix(fn, "dup", dup, dtype, rows, cols, dup_ld, true)) return e;
        a.up_codes = const_cast<int8_t*>(up_codes);
        a.up_exponents = const_cast<uint8_t*>(up_exponents);
        a.dup = dup;
        a.dup_ld = dup_ld;
    } else if (dup) {
        return fail(ZERO_EINVAL, "%s: dup without a checkpoint of up", fn);
    }
    if (again_codes || again_exponents) {
        if (int e = check_saved(fn, "act(x)", again_codes, again_exponents)) return e;
        a.again_codes = again_codes;
        a.again_exponents = again_exponents;
    }
    return run_act(fn, a, 1, stream);
}

namespace {
int weight_plan(const char* fn, int64_t rows, int64_t outs, int64_t cols, zf::WeightGrad* a, int64_t* bytes) {
    if (rows < 0 || outs < 0 || cols < 0) return fail(ZERO_EINVAL, "%s: negative size", fn);
    if (rows > (int64_t)1 << 34 || outs > kMaxCols || cols > kMaxCols || outs * cols > (int64_t)1 << 38)
        return fail(ZERO_ERANGE, "%s: more than 2^34 rows, 2^24 columns or 2^38 weights", fn);
    memset(a, 0, sizeof *a);
    a->rows = rows;
    a->outs = outs;
    a->cols = cols;
    a->pitch = (cols + 31) / 32 * 32;
    zf::plan_weight_grad(*a);
    *bytes = (a->tiles - a->whole_tiles) * a->splits * a->tile * a->tile * 4;
    return ZERO_OK;
}
}  // namespace

int zero_weight_grad8_workspace(int64_t rows, int64_t outs, int64_t cols, int64_t* bytes) {
    const char* fn = "zero_weight_grad8_workspace";
    if (!bytes) return fail(ZERO_EINVAL, "%s: NULL bytes", fn);
    zf::WeightGrad a;
    if (int e = weight_plan(fn, rows, outs, cols, &a, bytes)) return e;
    return ok();
}

int zero_weight_grad8(const void* dy, int32_t dy_dtype, int64_t dy_ld, int64_t rows, int64_t outs,
                      const int8_t* codes, const uint8_t* exponents, int64_t cols, void* grad,
                      int32_t grad_dtype, uint32_t flags, void* workspace, int64_t workspace_bytes,
                      void* stream) {
    const char* fn = "zero_weight_grad8";
    if (dy_dtype != ZERO_F16 && dy_dtype != ZERO_BF16)
        return fail(ZERO_EINVAL, "%s: dy_dtype must be fp16 or bf16", fn);
    if (!valid_dtype(grad_dtype)) return fail(ZERO_EINVAL, "%s: bad grad_dtype %d", fn, grad_dtype);
    if (flags & ~ZERO_ACCUMULATE) return fail(ZERO_EINVAL, "%s: unknown flags", fn);
    zf::WeightGrad a;
    int64_t need;
    if (int e = weight_plan(fn, rows, outs, cols, &a, &need)) return e;
    const bool accumulate = flags & ZERO_ACCUMULATE;
    if (outs == 0 || cols == 0 || (rows == 0 && accumulate)) return ok();
    if (!grad) return fail(ZERO_EINVAL, "%s: NULL grad", fn);
    if (!aligned(grad, esize(grad_dtype))) return fail(ZERO_EALIGN, "%s: grad not aligned to its element size", fn);
    if (rows > 0) {
        if (int e = check_matrix(fn, "dy", dy, dy_dtype, rows, outs, dy_ld, false)) return e;
        if (int e = check_saved(fn, "x", codes, exponents)) return e;
    }
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(ZERO_EINVAL, "%s: the workspace needs %lld bytes", fn, (long long)need);
    if (need > 0 && !aligned(workspace, 16)) return fail(ZERO_EALIGN, "%s: workspace not 16-byte aligned", fn);
    a.dy = dy;
    a.dy_ld = dy_ld;
    a.codes = codes;
    a.exponents = exponents;
    a.grad = grad;
    a.grad_dtype = grad_dtype;
    a.accumulate = accumulate;
    a.partials = need > 0 ? static_cast<float*>(workspace) : nullptr;
    const int e = zf::launch_weight_grad(a, dy_dtype, stream);
    if (e) return hip_fail(e, fn);
    return ok();
}

}  // extern "C"
