// zf_launch.h -- internal interface between the C-ABI layer (zeroflat_api.cpp)
// and the gfx950 kernels (zeroflat_kernels.hip).  Arguments reaching these
// launchers have been validated; they only pick a kernel variant and launch.
#pragma once

#include <stdint.h>

#include "zeroflat.h"

namespace zf {

// Reduce (n_ranks buffers) or statistics-only (n_ranks == 1, red_out == null)
// over [0, n) of each buffer (pointers already offset to the rank's slice).
struct ReduceLaunch {
    const void* bufs[ZERO_MAX_RANKS];
    int32_t n_ranks;
    int32_t dtype;   // zero_dtype_t of the inputs
    int32_t op;      // zero_reduce_op_t
    int32_t vec;     // 1: vector path (every pointer allows quad accesses, from
                     // element `head` on for the inputs)
    int32_t head;    // vector path: elements 0 .. head-1 precede the inputs' first
                     // 128-byte line boundary (0..63; the output is 16-byte
                     // aligned at element 0)
    int64_t n;
    float* red_out;  // may be null
    int32_t accumulate;     // 1: red_out += reduce (red_out is read, then written)
    int32_t block;          // INT8 payload only: elements per scale
    int32_t block_shift;    // log2(block) if a power of two, else -1
    zero_step_state_t* st;  // may be null
    double* partials;       // per-block partial sums of the statistics (st set):
                            // st->partials, or the library's scratch
};
int launch_reduce_stats(const ReduceLaunch& a, void* stream);
// The same launch with the statistics' partial sums in the library's own
// device scratch (one array per device, found on the first call on a device)
// instead of the state's table; the state then needs only its header.
int launch_reduce_noalloc(ReduceLaunch& a, void* stream);
// The quantised-gradient reduce: bufs[2k] = rank k's INT8 codes, bufs[2k+1]
// its fp32 block scales (n_ranks <= ZERO_MAX_RANKS / 2).
int launch_reduce_q8(const ReduceLaunch& a, void* stream);

struct AdamLaunch {
    const void* g;
    int32_t gdtype;
    int32_t pdtype;
    float* p;
    float* m;
    float* v;
    int64_t n;
    void* lp;        // All-Gather slot, already offset
    int8_t* q;       // INT8 slot, already offset (or null)
    float* qs;       // scales of the slot, already offset
    int32_t vec;     // 1: vector path allowed
    uint32_t flags;
    float b1, c1, b2, c2, lr, wdf, eps;
    double beta1, beta2, max_norm;
    zero_step_state_t* st;
};
int launch_adamw(const AdamLaunch& a, void* stream);

struct QuantLaunch {
    const void* x;
    int32_t dtype;
    int32_t vec;     // 2: eight elements per lane (x 16-byte, q 8-byte aligned);
                     // 1: quad tiles (x 8-byte, q 4-byte aligned); 0: element-wise
    int64_t n;
    int8_t* q;
    float* qs;
};
int launch_quant(const QuantLaunch& a, void* stream);

// Dequantise n_slots INT8 slots of slot_numel codes into the flat buffer.
struct DequantLaunch {
    const int8_t* q;
    const float* qs;
    void* out;
    int32_t out_dtype;
    int32_t block;
    int32_t n_slots;
    int32_t vec;     // 1: slot_numel % 4 == 0 and every pointer allows quad accesses
    int64_t slot_numel;
};
int launch_dequant(const DequantLaunch& a, void* stream);

// The step over a list of tensors (zeroflat_multi.hip).  One table entry per
// tensor, in the plan's device image.
struct MultiEntry {
    const void* grad;
    void* param;         // 16-bit copy, or null
    int64_t numel;
    int64_t row0;        // first row of the arenas
    double lr_mult;
    double decay_mult;
    int32_t tile0;       // first tile of the update
    int32_t span0;       // first span of the statistics
    int32_t n_spans;
    int32_t reserved;
};
static_assert(sizeof(MultiEntry) == 64, "the table's entries are 64 bytes");

// A list is short up to kMultiShortSpans spans of its statistics, of which a
// tensor that is not empty has one at least: its update folds them itself, which
// takes a launch less.  Whole steps with the limit at
// 512, 1024 and 2048 spans, us: 10 tensors of 8e6 elements in all, 32-bit
// states 52, 52, 48, 8-bit 35, 35, 33; 700 of 4e6 34, 34, 28 and 23, 23, 22.
// Lists on either side of it: 2,000 and 2,100 tensors of 64 elements 12.1 and
// 14.7, of 900 elements 20.9 and 24.7 (32-bit; 8-bit 12.1 and 13.9, 15.8 and
// 19.7).
constexpr int64_t kMultiShortSpans = 2048;
// Rows of one wave's tile of the update.  Fewer rows shorten a wave's chain of
// loads and arithmetic; more keep more bytes in flight per wave.  1, 2 and 4
// rows, us: 20,000 elements 7.5, 8.1, 9.2 (32-bit states) and 7.4, 7.9, 8.7
// (8-bit); 1.05e6 10.3, 10.7, 11.8 and 9.7, 9.5, 10.4; 4e6 25.9, 26.1, 29.2
// and 22.3, 20.0, 20.6; 3e7 144, 139, 139 and 88, 81, 82.
constexpr int kMultiRowsLong = 4, kMultiRowsShort = 2, kMultiRowsTiny = 1;
constexpr int64_t kMultiTinyRows = 2048;   // a short list of at most so many rows is tiny

// the scalars of a step state
struct MultiState {
    double sumsq, remote_sumsq, beta1_pow, beta2_pow;
    float loss_scale, min_scale;
    int32_t overflow, remote_overflow, dynamic, window, good_steps, step;
};
// a step's scalars, formed from them
struct MultiScalars {
    double lr, lr_bc1, wd, norm;    // lr, lr / (1 - beta1^t), weight decay
    float inv, coef, bc1, bc2, rs;
    uint32_t key;
    int32_t skip;
};

struct MultiNormLaunch {
    const MultiEntry* entries;
    const int32_t* span_tensor;
    double* tensor_sumsq;
    double* partials;
    MultiState* snapshot;   // null, or where the pass leaves the state's scalars
    zero_step_state_t* st;
    int64_t span;
    int32_t n_tensors, n_spans;
    int32_t keep_spans;     // the first spans, read again by the update: kept in the caches
    int32_t dtype;
    int32_t reset;
};
int launch_multi_norm(const MultiNormLaunch& a, void* stream);

struct MultiStep {
    MultiScalars* scalars;      // where the step's scalars go
    zero_step_state_t* st;
    double lr, wd, beta1, beta2, max_norm;
    uint32_t seed;
    int32_t advance;            // 1: the loss scaler and the counters move on
};
struct MultiAdamLaunch {
    const MultiEntry* entries;
    const int32_t* tile_tensor;
    const MultiScalars* scalars;
    float* p;
    void* m;
    void* v;
    float* ms;
    float* vs;
    int32_t n_tiles;
    int32_t tile_rows;          // kMultiRowsLong, -Short or -Tiny
    int32_t gdtype, pdtype, bits;
    float b1, c1, b2, c2, eps;
};
// norm: null, or the list's statistics, taken first
int launch_multi_step(const MultiAdamLaunch& a, const MultiNormLaunch* norm, const MultiStep& step,
                      void* stream);

// ZeRO-Offload (zeroflat_offload.cpp).  The host update over host arrays:
// *skipped = 1 (and nothing written) when the state says overflow.
int offload_adam_host(const void* g, int32_t gdt, float* p, float* m, float* v, int64_t n,
                      void* lp, int32_t pdt, const zero_adamw_hparams_t& hp,
                      const zero_step_state_t& st, int32_t n_threads, int* skipped);
// The pipelined step: gradient chunks device->host, host update, 16-bit
// parameter chunks host->device into the slot, then the device finalize.
// Blocks the calling thread until every copy has completed.
struct OffloadLaunch {
    const void* d_grad;
    int32_t gdtype;
    int32_t pdtype;
    int64_t n;
    float* h_p;
    float* h_m;
    float* h_v;
    void* h_grad;     // pinned staging, n gradient elements
    void* h_lp;       // pinned staging, n 16-bit parameters
    void* d_slot;     // the All-Gather slot, already offset
    int64_t chunk;
    int32_t n_threads;
    zero_step_state_t* st;
};
int offload_step(const OffloadLaunch& a, const zero_adamw_hparams_t& hp, void* stream);

const char* hip_error_string(int err);

}  // namespace zf
