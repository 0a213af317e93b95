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

// The embedding (zeroflat_embed.hip).
constexpr int kEmbedInt8 = 3;            // a table's type beside zero_dtype_t: the INT8 payload
constexpr int kEmbedFew = 2048;          // tokens whose gradient needs no sort, at most
constexpr int kEmbedSortTile = 1024;     // tokens of one block of the sort
// Zeros that a launch of the sort writes beside it, as many as its latency hides: 0, 20,
// 40 and 80 MiB a launch, us: 4096 x 4096 into 32000 bf16 rows 80, 67, 63, 65; 16384 x 4096
// 101, 91, 90, 93; 30011 x 1001 into 50021 fp32 rows 94, 81, 75, 77; 16384 x 2048 into
// 131072 251, 236, 227, 220.  Where tokens name most rows they are written in vain: 131072
// x 512 into 32000 fp32 rows 75, 83, 82, 82.
constexpr int64_t kEmbedZeroBytes = 40 << 20;
// Blocks of the sort that sum the counts before theirs themselves; more have a launch
// between.  So and with it, us, n x 64 added: 16384 tokens 32, 36; 65536 44, 45; 131072 (128
// blocks) 56, 52; 262144 81, 66; 2^20 223, 145.
constexpr int kEmbedScanBlocks = 128;
constexpr int kEmbedTile = 128;          // sorted positions of a block of the sums, at most
constexpr int kEmbedBatch = 8;           // rows that a wave of the sums has in flight

// Whether a call's output of so many bytes goes past the caches: from half the
// memory-side cache on, where its reader would not find the beginning any more.
// Written and then copied, cached and past the caches, us: embedding rows 64 MiB 44, 50,
// 96 MiB 65, 72, 128 MiB 101, 99, 256 MiB 201, 195; an activation's gradient 47, 52; 74,
// 81; 115, 110; 213, 215.  Written alone, 128 MiB of rows from an INT8 payload 55, 31: the
// payload stays cached.
constexpr int64_t kStreamBytes = (int64_t)128 << 20;
inline int streams(int64_t bytes) { return bytes >= kStreamBytes; }

// n / d by a product (see zf_vec.h)
struct Div {
    uint32_t d, m, s;
};

struct EmbedLookup {
    const void* tokens;
    const void* table;      // INT8: the payload's codes
    const float* scales;    // INT8 only, as the fields below it
    int64_t elem_offset, slot_numel, slot_blocks;
    void* out;
    int64_t out_ld, first, vocab, dim;
    Div per_row;            // groups of eight columns in a row
    uint32_t groups;
    int32_t stream;         // 1: the output goes past the caches
    int32_t wide;           // 1: 64-bit tokens
    float scale;
};
struct EmbedLookupLaunch {
    EmbedLookup args;
    int64_t n_tokens, dim;
    int32_t table_dtype, out_dtype;
};
int launch_embed_lookup(const EmbedLookupLaunch& a, void* stream);

struct EmbedSort {
    const void* tokens;
    int64_t n_tokens, first, padding, vocab;
    const uint32_t* keys_in;
    const int32_t* places_in;
    uint32_t* keys_out;
    int32_t* places_out;
    uint32_t* hist;
    uint32_t* flags;        // a byte per row, 1 where a token names it; null: not asked for
    int64_t flag_words;
    char* grad;             // zeros go to bytes [zero_first, zero_last) of it
    int64_t zero_first, zero_last;
    int32_t stream;         // 1: they go past the caches
    int32_t wide, has_padding, passes, pass, digit_bits, blocks, scanned;
};
struct EmbedSum {
    const uint32_t* keys;
    const int32_t* places;
    const uint32_t* flags;
    const void* dy;
    void* grad;
    float* partials;        // two fp32 rows of `pitch` per tile: a run from before, a run that goes on
    int64_t n_tokens, vocab, dim, dy_ld, pitch, tiles, chunks, sum_blocks;
    int64_t zero_from;      // the first row that may need zeros yet
    Div row_chunks;         // 16-byte parts of a row
    int32_t zero_rows;      // rows of one block that writes zeros
    int32_t tile;           // sorted positions of one tile
    int32_t accumulate;
    int32_t stream;         // 1: the gradient goes past the caches
    float scale;
};
struct EmbedGradLaunch {
    EmbedSort sort;
    EmbedSum sum;
    void* workspace;
    int32_t dy_dtype, grad_dtype;
};
int launch_embed_grad(const EmbedGradLaunch& a, void* stream);

// Few tokens find one another by comparing, in one launch: n * n comparisons for
// every 512 columns.  In us, and by the sort with its five launches at least (zipf tokens,
// added to 32000 bf16 rows): 512 x 256 8, 26; 512 x 4096 10, 25; 1024 x 1024 10, 26;
// 2048 x 256 17, 29; beyond the limit 1024 x 4096 27, 27; 2048 x 1024 29, 28; 4096 x 256
// 31, 30.  One token 2048 times: 30, 26.
inline bool embed_few(int64_t n, int64_t dim) {
    const int64_t chunks = dim > 512 ? (dim + 511) / 512 : 1;
    return n <= kEmbedFew && n * n * chunks <= (int64_t)kEmbedFew * kEmbedFew;
}

// The parts of its workspace, as byte offsets.
struct EmbedWorkspace {
    int64_t keys[2], places[2], hist, flags, partials, bytes;
    int64_t tiles, pitch;
    int32_t tile;
};
// The tile: long enough that its partial rows (fp32, two at most) are little beside
// its rows, short enough that few tokens spread over the chip.  128 and 32 positions,
// us: 5000 x 512 37, 30; 16384 x 512 41, 34; 32768 x 512 44, 42; 16384 x 2048 59, 58;
// 65536 x 512 57, 59; 131072 x 1024 117, 118.
inline EmbedWorkspace embed_workspace(int64_t n, int64_t vocab, int64_t dim) {
    EmbedWorkspace w{};
    if (embed_few(n, dim)) return w;
    const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    w.tile = n * ((dim + 511) / 512) >= 65536 ? kEmbedTile : 32;
    w.tiles = (n + w.tile - 1) / w.tile;
    w.pitch = (dim + 7) / 8 * 8;
    int64_t at = 0;
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = at;
        at += up(n * 4);
        w.places[k] = at;
        at += up(n * 4);
    }
    w.hist = at;
    at += up(((n + kEmbedSortTile - 1) / kEmbedSortTile + 1) * 256 * 4);
    w.flags = at;
    at += up(vocab);
    w.partials = at;
    at += up(w.tiles * 2 * w.pitch * 4);
    w.bytes = at;
    return w;
}

// Activations kept in 8 bits (zeroflat_act.hip).  Forward: x, and up where it is
// gated, into their checkpoints, y = act(x) [* up].  Backward: x is dy, y its
// gradient of x.  kind < 0: no function, the checkpoint alone, or restored to y.
struct ActLaunch {
    const void* x;
    const void* up;
    void* y;
    void* dup;
    int8_t* codes;
    uint8_t* exponents;
    int8_t* up_codes;            // null: not gated
    uint8_t* up_exponents;
    int8_t* again_codes;         // backward: the checkpoint of act(x) [* up], or null
    uint8_t* again_exponents;
    int64_t rows, cols, x_ld, up_ld, y_ld, dup_ld;
    Div per_row;                 // groups of eight columns in a checkpoint's row
    uint32_t groups;
    int32_t stream;              // 1: y and dup go past the caches
    int32_t dtype, kind;
    int32_t least;               // the least exponent that a checkpoint takes
};
int launch_act(const ActLaunch& a, int backward, void* stream);

// A weight gradient (zeroflat_wgrad.hip).
struct WeightGrad {
    const void* dy;
    const int8_t* codes;
    const uint8_t* exponents;
    void* grad;
    float* partials;             // the shares' sums, a whole tile each
    int64_t rows, outs, cols, pitch, dy_ld;
    int64_t share;               // rows of a share
    int64_t tiles, tiles_o, tiles_i;
    int64_t whole_tiles;         // tiles that one block sums; the others are shared by `splits` blocks
    int32_t tile, splits, grad_dtype, accumulate;
};
int launch_weight_grad(const WeightGrad& a, int dtype, void* stream);
// The tile and the split, which the sizes alone fix.
void plan_weight_grad(WeightGrad& a);

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
