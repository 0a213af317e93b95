// zeroflat_embed.hip -- gfx950 (MI355X, CDNA4, wave64) kernels of the embedding:
//   embed_lookup_kernel   rows of the table by token, scaled; the table a view
//                         of the flat parameter, or the gathered INT8 payload
//   embed_few_kernel      the gradient of up to kEmbedFew tokens, in one launch
//   embed_hist_kernel, embed_scan_kernel, embed_scatter_kernel
//                         the positions of more, sorted by token, stable
//   embed_sum_kernel      the gradient's rows summed over runs of equal tokens
//   embed_join_kernel     the runs that cross tiles
//
// The gradient of row v is the sum of dy's rows at the tokens equal to v.  Added
// by atomics its roundings would depend on the order of arrival, and a frequent
// token's row would be one address for the whole chip.  Sorted, the positions
// are cut into tiles of one length whatever the tokens are, so that every wave
// has the same work; a run inside a tile is summed in registers and LDS and written
// once, and one that crosses tiles leaves an fp32 partial row per tile, which
// the join adds in order.  Few tokens need no sort: the wave of a token's first
// position finds the others by comparing.  Every sum's order is fixed by the
// tokens alone.
//
// Bound by memory: dy once, the written rows once.  The sort's launches move next
// to nothing and take 23 us; where every row is written, they write zeros
// meanwhile, to rows that a token names too (those are written again), and the
// sums' launch to the others that are left: 16384 x 4096 into 32000 bf16 rows takes
// 90 us, 4.4 TB/s (100 with all zeros in the sums' launch).
#include "zf_vec.h"

namespace zf {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 256;             // digits of up to 8 bits
constexpr int kRounds = kEmbedSortTile / kThreads;
constexpr int kChunk = 512;            // columns of one wave: eight per lane

#define ZF_CONST __attribute__((address_space(4)))
// Read-only while the kernel runs: wave-uniform reads stay scalar.
template <typename T>
__device__ __forceinline__ const ZF_CONST T* as_const(const T* p) {
    return (const ZF_CONST T*)(uintptr_t)p;
}

__device__ __forceinline__ int64_t token_at(const void* tokens, int wide, int64_t i) {
    return wide ? static_cast<const int64_t*>(tokens)[i] : (int64_t)static_cast<const int32_t*>(tokens)[i];
}
// The token's row of the table, or `vocab` if it has none here.
__device__ __forceinline__ uint32_t row_of(int64_t token, int64_t first, uint32_t vocab) {
    return token >= first && (uint64_t)(token - first) < vocab ? (uint32_t)(token - first) : vocab;
}

// ---------------------------------------------------------------- lookup
// One group of eight columns of one token's row per lane.  Bound by memory: the
// row and the output, once each: 16384 rows of 4096 from the INT8 payload into bf16 in 31
// us, 6.5 TB/s; one row by the launch, 2 us of the GPU and 5.7 of the host.
template <int TT, int TO>
__global__ __launch_bounds__(kThreads) void embed_lookup_kernel(EmbedLookup a) {
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= a.groups) return;
    const uint32_t t = div_by(g, a.per_row);
    const uint32_t col = (g - t * a.per_row.d) * 8;
    const int n = (int)min((uint32_t)8, (uint32_t)a.dim - col);
    const uint32_t row = row_of(token_at(a.tokens, a.wide, t), a.first, (uint32_t)a.vocab);
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (row < (uint32_t)a.vocab) {
        const int64_t at = (int64_t)row * a.dim + col;
        if constexpr (TT != kEmbedInt8) {
            load8<TT>(a.table, at, n, x);
        } else {
            // element `at` of the table is code at + elem_offset of the payload:
            // slot s, place i within it, block i / 256 of the slot's scales
            const int8_t* q = static_cast<const int8_t*>(a.table);
            int64_t e = at + a.elem_offset;
            const int64_t s = e / a.slot_numel, i = e - s * a.slot_numel;
            const float* sc = a.scales + s * a.slot_blocks;
            if (n >= 8 && i + 8 <= a.slot_numel) {
                const v2u c = *reinterpret_cast<const v2u_any*>(q + e);
                const int64_t b = i >> 8;
                const int left = 256 - (int)(i & 255);
                const float s0 = sc[b], s1 = left < 8 ? sc[b + 1] : s0;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    x[k] = (float)(int8_t)(c[k / 4] >> (8 * (k % 4))) * (k < left ? s0 : s1);
            } else {
                for (int k = 0; k < n; ++k, ++e) {
                    const int64_t sk = e / a.slot_numel;
                    x[k] = (float)q[e] * a.scales[sk * a.slot_blocks + ((e - sk * a.slot_numel) >> 8)];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] *= a.scale;
    }
    store8<TO>(a.out, (int64_t)t * a.out_ld + col, n, x, a.stream);
}

// ---------------------------------------------------------------- sort
// Exclusive sum over the block's threads of 64-lane waves, in thread order.
template <int WAVES>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* lds, uint32_t* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t s = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    if (lane == 63) lds[wave] = s;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const uint32_t v = lds[w];
        if (w < wave) before += v;
        all += v;
    }
    __syncthreads();
    *total = all;
    return before + s - x;
}

// The lanes of the wave that hold the same digit as this one.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, int bits, bool live) {
    uint64_t m = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const uint64_t v = __ballot((d >> b) & 1);
        m &= (d >> b) & 1 ? v : ~v;
    }
    return m;
}

__device__ __forceinline__ uint32_t key_at(const EmbedSort& a, int64_t i) {
    const int64_t token = token_at(a.tokens, a.wide, i);
    return token == a.padding && a.has_padding ? (uint32_t)a.vocab : row_of(token, a.first, (uint32_t)a.vocab);
}

// Zeros over [first, last) bytes of a gradient, both multiples of two: 16 KiB a
// block, 16 bytes a lane and store at any address.
constexpr int64_t kZeroBlock = 16384;
__device__ __forceinline__ void zero_bytes(char* grad, int64_t first, int64_t last, int64_t block, int stream) {
    const int64_t from = first + block * kZeroBlock, to = min(last, from + kZeroBlock);
    for (int64_t at = from + threadIdx.x * 16; at < to; at += kThreads * 16) {
        v4u_any* p = reinterpret_cast<v4u_any*>(grad + at);
        if (at + 16 <= to && stream) {
            ZF_APART;
            __builtin_nontemporal_store(v4u_any{0, 0, 0, 0}, p);
            ZF_APART;
        } else if (at + 16 <= to) *p = v4u_any{0, 0, 0, 0};
        else
            for (int64_t b = at; b < to; b += 2) *reinterpret_cast<uint16_t*>(grad + b) = 0;
    }
}

// Zeros to the rows from v0 on, a.zero_rows of them, that `hit` does not name: 16 bytes a
// lane and store, whole lines in turn whatever the rows' length.  (Rows by waves, eight
// columns a lane, wrote 1 GiB in 468 us behind few tokens and 414 behind the sort.)
constexpr int64_t kZeroRowsBytes = 32768;
template <int TG, int THREADS, typename Hit>
__device__ __forceinline__ void zero_rows(const EmbedSum& a, int64_t v0, int64_t vocab, Hit hit) {
    using T = typename Elem<TG>::type;
    constexpr int wide = 16 / sizeof(T);
    const uint32_t all = (uint32_t)min((int64_t)a.zero_rows, vocab - v0) * a.row_chunks.d;
    for (uint32_t q = threadIdx.x; q < all; q += THREADS) {
        const uint32_t r = div_by(q, a.row_chunks);
        const int64_t col = (int64_t)(q - r * a.row_chunks.d) * wide;
        if (hit(r)) continue;
        T* p = static_cast<T*>(a.grad) + (v0 + r) * a.dim + col;
        if (col + wide <= a.dim && a.stream) {
            ZF_APART;
            __builtin_nontemporal_store(v4u_any{0, 0, 0, 0}, reinterpret_cast<v4u_any*>(p));
            ZF_APART;
        } else if (col + wide <= a.dim) {
            *reinterpret_cast<v4u_any*>(p) = v4u_any{0, 0, 0, 0};
        } else {
            for (int64_t c = col; c < a.dim; ++c) *p++ = T(0);
        }
    }
}

// One pass, first half: how many of each digit a block of
// kEmbedSortTile items holds.  The first pass reads the tokens and clears the
// rows' marks.
__global__ __launch_bounds__(kThreads) void embed_hist_kernel(EmbedSort a) {
    __shared__ uint32_t count[kBins];
    if (blockIdx.x >= (uint32_t)a.blocks) {
        zero_bytes(a.grad, a.zero_first, a.zero_last, blockIdx.x - a.blocks, a.stream);
        return;
    }
    count[threadIdx.x] = 0;
    if (a.pass == 0 && a.flags)
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < a.flag_words;
             i += (int64_t)a.blocks * kThreads)
            a.flags[i] = 0;
    __syncthreads();
    const uint32_t mask = (1u << a.digit_bits) - 1, shift = a.pass * a.digit_bits;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t i = (int64_t)blockIdx.x * kEmbedSortTile + r * kThreads + threadIdx.x;
        if (i < a.n_tokens) {
            const uint32_t key = a.pass == 0 ? key_at(a, i) : a.keys_in[i];
            atomicAdd(&count[(key >> shift) & mask], 1u);      // counts: any order gives the same
        }
    }
    __syncthreads();
    a.hist[(int64_t)blockIdx.x * kBins + threadIdx.x] = count[threadIdx.x];
}

// Lists of more than kEmbedScanBlocks blocks: each digit's counts summed over
// the blocks before, one block per digit, totals behind the table.
__global__ __launch_bounds__(kThreads) void embed_scan_kernel(EmbedSort a) {
    __shared__ uint32_t sums[kWaves];
    const int d = blockIdx.x;
    uint32_t base = 0;
    for (int b0 = 0; b0 < a.blocks; b0 += kThreads) {
        const int b = b0 + (int)threadIdx.x;
        uint32_t all;
        const uint32_t c = b < a.blocks ? a.hist[(int64_t)b * kBins + d] : 0;
        const uint32_t at = block_scan<kWaves>(c, sums, &all);
        if (b < a.blocks) a.hist[(int64_t)b * kBins + d] = base + at;
        base += all;
    }
    if (threadIdx.x == 0) a.hist[(int64_t)a.blocks * kBins + d] = base;
}

// Second half of a pass: every item to its place.  Up to kEmbedScanBlocks
// blocks each block sums the table itself, which saves the launch between.
__global__ __launch_bounds__(kThreads) void embed_scatter_kernel(EmbedSort a) {
    __shared__ uint32_t count[kWaves][kBins];
    __shared__ uint32_t sums[kWaves];
    if (blockIdx.x >= (uint32_t)a.blocks) {
        zero_bytes(a.grad, a.zero_first, a.zero_last, blockIdx.x - a.blocks, a.stream);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t before = 0, total = 0;
    if (a.scanned) {
        before = a.hist[(int64_t)blockIdx.x * kBins + threadIdx.x];
        total = a.hist[(int64_t)a.blocks * kBins + threadIdx.x];
    } else {
        // 32 loads at a time: one after the other they took half the kernel
        for (int b0 = 0; b0 < a.blocks; b0 += 32) {
            uint32_t c[32];
#pragma unroll
            for (int k = 0; k < 32; ++k)
                c[k] = b0 + k < a.blocks ? a.hist[(int64_t)(b0 + k) * kBins + threadIdx.x] : 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
                total += c[k];
                if (b0 + k < (int)blockIdx.x) before += c[k];
            }
        }
    }
#pragma unroll
    for (int w = 0; w < kWaves; ++w) count[w][threadIdx.x] = 0;
    uint32_t all;
    const uint32_t base = before + block_scan<kWaves>(total, sums, &all);
    const uint32_t mask = (1u << a.digit_bits) - 1, shift = a.pass * a.digit_bits;
    uint32_t key[kRounds], place[kRounds], rank[kRounds];
    const int64_t first = (int64_t)blockIdx.x * kEmbedSortTile + wave * 64 * kRounds + lane;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int64_t i = first + r * 64;
        const bool live = i < a.n_tokens;
        key[r] = !live ? 0 : a.pass == 0 ? key_at(a, i) : a.keys_in[i];
        place[r] = !live ? 0 : a.pass == 0 ? (uint32_t)i : (uint32_t)a.places_in[i];
        if (a.pass == 0 && a.flags && live && key[r] < (uint32_t)a.vocab)
            reinterpret_cast<uint8_t*>(a.flags)[key[r]] = 1;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const bool live = first + r * 64 < a.n_tokens;
        const uint32_t d = (key[r] >> shift) & mask;
        const uint64_t m = same_digit(d, a.digit_bits, live);
        const int below = __popcll(m & ((1ull << lane) - 1));
        const uint32_t had = live ? count[wave][d] : 0;
        rank[r] = had + below;
        // a wave's own counts, and its LDS operations keep their order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (live && below == 0) count[wave][d] = had + __popcll(m);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    uint32_t at = base;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t c = count[w][threadIdx.x];
        count[w][threadIdx.x] = at;
        at += c;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        if (first + r * 64 < a.n_tokens) {
            const uint32_t to = count[wave][(key[r] >> shift) & mask] + rank[r];
            a.keys_out[to] = key[r];
            a.places_out[to] = (int32_t)place[r];
        }
    }
}

// ---------------------------------------------------------------- sums
// Columns col .. col + 7 of a row's sum into the gradient; of a row's last columns a
// lane has eight that end with the row, and writes those from `skip` on.
template <int TG>
__device__ __forceinline__ void write_row(const EmbedSum& a, uint32_t row, int64_t col, int skip, int n,
                                          float (&acc)[8]) {
    const int64_t at = (int64_t)row * a.dim + col;
    float y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = acc[k] * a.scale;
    if (skip == 0 && n >= 8) {
        if (a.accumulate) {
            const Raw8<TG> old = fetch8<TG>(a.grad, at);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] += element<TG>(old, k);
        }
        store8<TG>(a.grad, at, 8, y, a.stream);
        return;
    }
    auto* p = static_cast<typename Elem<TG>::type*>(a.grad) + at;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k >= skip && k < n) p[k] = from_f32<TG>(a.accumulate ? y[k] + to_f32<TG>(p[k]) : y[k]);
}

// The eight columns that a lane loads for its group at `col`: those, or the row's
// last eight, of which it owns the ones from `skip` on; of a row of less than eight
// the first n.
struct Window {
    int64_t col;
    int skip, n;
};
__device__ __forceinline__ Window window_at(int64_t col, int64_t dim) {
    const int64_t w = max((int64_t)0, min(col, dim - 8));
    return Window{w, (int)min((int64_t)8, col - w), (int)min((int64_t)8, dim - w)};
}
template <int TD, bool NARROW>
__device__ __forceinline__ Raw8<TD> fetch_row(const EmbedSum& a, int64_t place, const Window& w) {
    if constexpr (!NARROW) {
        return fetch8<TD, true>(a.dy, place * a.dy_ld + w.col);
    } else {
        const auto* p = static_cast<const typename Elem<TD>::type*>(a.dy) + place * a.dy_ld;
        Raw8<TD> r;
        r.lo = r.hi = v4u{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < 7; ++k) {
            const auto x = p[min(k, w.n - 1)];             // columns behind the last repeat it
            if constexpr (TD == ZERO_F32) (k < 4 ? r.lo : r.hi)[k % 4] = __float_as_uint(x);
            else r.lo[k / 2] |= (uint32_t)x << (16 * (k & 1));
        }
        return r;
    }
}

// A block takes 512 columns of a tile of sorted positions, a wave a quarter of it.  A
// run that crosses quarters is added up in LDS; one that crosses tiles leaves the
// tile's share in its first partial row (it began before) or its second (it begins
// here and goes on).  Blocks behind them write zeros to the rows that no token
// names, 32 KiB each.
template <int TD, int TG, bool NARROW>
__global__ __launch_bounds__(kThreads) void embed_sum_kernel(EmbedSum a) {
    __shared__ float heads[kWaves][kChunk];
    __shared__ int32_t state[kWaves];                      // of a quarter, as bits:
    constexpr int kHead = 1, kThrough = 2, kTail = 4;      // a run from before; the only one, and it goes on; one that begins and goes on
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    if (blockIdx.x >= (uint32_t)a.sum_blocks) {
        const int64_t v0 = a.zero_from + (int64_t)(blockIdx.x - a.sum_blocks) * a.zero_rows;
        const uint8_t* named = reinterpret_cast<const uint8_t*>(a.flags) + v0;
        zero_rows<TG, kThreads>(a, v0, a.vocab, [&](uint32_t r) { return as_const(named)[r] != 0; });
        return;
    }
    const int64_t tile = blockIdx.x / (uint32_t)a.chunks;
    const int64_t col = (blockIdx.x - tile * a.chunks) * kChunk + lane * 8;
    const Window w = window_at(col, a.dim);
    const int quarter = a.tile / kWaves;
    const int64_t base = tile * a.tile + wave * quarter;
    const int len = (int)max((int64_t)0, min((int64_t)quarter, a.n_tokens - base));
    // lane j holds the quarter's j-th key and place, lane 62 the key before, lane 63 the one behind
    static_assert(kEmbedTile / kWaves <= 62, "two lanes are left");
    const uint32_t none = (uint32_t)a.vocab;
    const int64_t at = lane == 62 ? base - 1 : lane == 63 ? base + len : base + min(lane, len - 1);
    const uint32_t key_here = at >= 0 && at < a.n_tokens ? a.keys[at] : none;
    const int32_t place_here = len > 0 ? a.places[base + min(lane, len - 1)] : 0;
    const auto key = [&](int j) { return (uint32_t)__builtin_amdgcn_readlane((int)key_here, j); };
    uint32_t cur = len > 0 ? key(0) : none;
    bool before = cur != none && key(62) == cur;           // the run began in an earlier quarter
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const auto keep = [&](float* to) {
        *reinterpret_cast<v4f*>(to + lane * 8) = v4f{acc[0], acc[1], acc[2], acc[3]};
        *reinterpret_cast<v4f*>(to + lane * 8 + 4) = v4f{acc[4], acc[5], acc[6], acc[7]};
    };
    const auto add = [&](const float* from) {
        const v4f x = *reinterpret_cast<const v4f*>(from + lane * 8), y = *reinterpret_cast<const v4f*>(from + lane * 8 + 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) { acc[c] += x[c]; acc[4 + c] += y[c]; }
    };
    const auto partial = [&](int which) {
        float* p = a.partials + (tile * 2 + which) * a.pitch + col;
        if (w.skip == 0) {
            *reinterpret_cast<v4f*>(p) = v4f{acc[0], acc[1], acc[2], acc[3]};
            *reinterpret_cast<v4f*>(p + 4) = v4f{acc[4], acc[5], acc[6], acc[7]};
        } else {
#pragma unroll
            for (int k = 1; k < 8; ++k)
                if (k >= w.skip) p[k - w.skip] = acc[k];
        }
    };
    int mine = 0;
    for (int j0 = 0; j0 < len && cur != none; j0 += kEmbedBatch) {
        // places behind the end repeat the last one: their rows are not used
        Raw8<TD> raw[kEmbedBatch];
#pragma unroll
        for (int j = 0; j < kEmbedBatch; ++j)
            raw[j] = fetch_row<TD, NARROW>(a, __builtin_amdgcn_readlane(place_here, j0 + j), w);
#pragma unroll
        for (int j = 0; j < kEmbedBatch; ++j) {
            if (j0 + j >= len) break;
            const uint32_t k = key(j0 + j);
            if (k != cur) {
                if (before) {
                    keep(heads[wave]);
                    mine = kHead;
                } else {
                    write_row<TG>(a, cur, w.col, w.skip, w.n, acc);
                }
                before = false;
                cur = k;
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] = 0.0f;
                if (cur == none) break;                    // the others are behind the last token
            }
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] += element<TD>(raw[j], c);
        }
    }
    if (cur != none) {
        const bool open = key(63) == cur;
        if (before) {
            keep(heads[wave]);
            mine = open ? kHead | kThrough : kHead;
        } else if (open) {
            mine |= kTail;                                 // (the sum stays in registers)
        } else {
            write_row<TG>(a, cur, w.col, w.skip, w.n, acc);
        }
    }
    if (lane == 0) state[wave] = mine;
    __syncthreads();
    if (mine & kTail) {
        // the quarters behind, as far as the run goes
        int u = wave + 1;
        for (; u < kWaves; ++u) {
            add(heads[u]);
            if (!(uniform(state[u]) & kThrough)) break;
        }
        if (u < kWaves) write_row<TG>(a, cur, w.col, w.skip, w.n, acc);
        else partial(1);
    }
    if (wave == 0 && (mine & kHead)) {
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = 0.0f;
        add(heads[0]);
        for (int u = 0; u < kWaves - 1 && (uniform(state[u]) & kThrough); ++u) add(heads[u + 1]);
        partial(0);
    }
}

// The block of tile t and 512 columns, if a run begins in t and ends in a later
// tile e: tail of t + heads of t+1 .. e.  Its waves take equal shares of the
// tiles, and the shares are added in order.
template <int TG>
__global__ __launch_bounds__(kThreads) void embed_join_kernel(EmbedSum a) {
    __shared__ float part[kWaves][kChunk];
    const int64_t tile = blockIdx.x;
    const int64_t base = tile * a.tile;
    const auto* keys = as_const(a.keys);
    const uint32_t k = keys[base + a.tile - 1];            // every tile but the last is full
    if (k == (uint32_t)a.vocab || keys[base + a.tile] != k) return;
    if (tile > 0 && keys[base] == k && keys[base - 1] == k) return;
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    // the last tile whose first key is k: 64 tiles a look, as the search is a chain of loads
    int64_t lo = tile + 1;
    for (;;) {
        const int64_t t = lo + 1 + lane;
        const uint64_t on = __ballot(t < a.tiles && a.keys[t * a.tile] == k);
        const int more = on == ~0ull ? 64 : __builtin_ctzll(~on);
        lo += more;
        if (more < 64) break;
    }
    const int64_t col = (int64_t)blockIdx.y * kChunk + lane * 8;
    const int n = (int)min((int64_t)8, a.dim - col);
    const int64_t many = lo - tile + 1, share = (many + kWaves - 1) / kWaves;
    const int64_t from = min(many, wave * share), to = min(many, from + share);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (n > 0) {
        for (int64_t j0 = from; j0 < to; j0 += kEmbedBatch) {
            // places behind the last repeat it: their rows are not used
            v4f x[kEmbedBatch], y[kEmbedBatch];
#pragma unroll
            for (int j = 0; j < kEmbedBatch; ++j) {
                const int64_t t = min(j0 + j, to - 1);
                const float* p = a.partials + ((tile + t) * 2 + (t == 0)) * a.pitch + col;
                x[j] = *reinterpret_cast<const v4f*>(p);
                y[j] = *reinterpret_cast<const v4f*>(p + 4);
            }
#pragma unroll
            for (int j = 0; j < kEmbedBatch; ++j)
                if (j0 + j < to)
#pragma unroll
                    for (int c = 0; c < 4; ++c) { acc[c] += x[j][c]; acc[4 + c] += y[j][c]; }
        }
    }
    *reinterpret_cast<v4f*>(&part[wave][lane * 8]) = v4f{acc[0], acc[1], acc[2], acc[3]};
    *reinterpret_cast<v4f*>(&part[wave][lane * 8 + 4]) = v4f{acc[4], acc[5], acc[6], acc[7]};
    __syncthreads();
    if (wave || n <= 0) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] += part[w][lane * 8 + c];
    write_row<TG>(a, k, col, 0, n, acc);
}

// The gradient of up to kEmbedFew tokens, without a sort.  The block holds every
// token's row and takes 512 columns; its wave w looks for the others of position
// 8 * block + w.  The wave that has the first of them sums them all in order, or, of
// more than kEmbedLong, leaves them to the whole block: each wave an eighth of the
// positions, the eighths added in order.  The blocks behind write zeros to the rows
// without a token.  Each looks at every token first and marks the named ones of its
// own rows: 16 rows a block, or what leaves kFewBlocks of them, two rounds of the
// chip, or the kEmbedFew that the marks have room for (beyond 3.1 million rows).  One
// launch, whose time is the chain of tokens, comparisons, rows.
// Measured, us: kEmbedLong 4, 8, 16 and 64, tokens by rank, 512 x 4096 added 11.6, 9.9, 9.6,
// 9.5, 2048 x 256 21.1, 19.2, 19.0, 17.1 (each token 64 times, 512 x 4096: 10.8, 10.5, 10.5,
// 10.0).  kFewBlocks 768, 1536 and four times that, 64 x 256 into 131072 bf16 rows 12.3, 11.9,
// 16.2; 512 x 256 20.0, 16.9, 21.4; 1024 x 1024 into 32000 28.0, 24.9, 29.0.
constexpr int kFewWaves = 8, kFewThreads = kFewWaves * 64, kEmbedLong = 16, kFewRows = 16, kFewBatch = 16;
constexpr int64_t kFewBlocks = 1536;

template <int TD, int TG, bool NARROW>
__global__ __launch_bounds__(kFewThreads) void embed_few_kernel(EmbedSort t, EmbedSum a) {
    __shared__ uint32_t keys[kEmbedFew];
    __shared__ uint16_t list[kFewWaves][kEmbedFew / kFewWaves];
    __shared__ float part[kFewWaves][kChunk];
    __shared__ uint32_t longs[kFewWaves];
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
    const int n = (int)t.n_tokens, blocks = (n + kFewWaves - 1) / kFewWaves;
    const uint32_t none = (uint32_t)t.vocab;
    const int64_t col = (int64_t)blockIdx.y * kChunk + lane * 8;
    if ((int)blockIdx.x >= blocks) {
        if (blockIdx.y) return;                            // whole rows
        const uint32_t v0 = (blockIdx.x - blocks) * (uint32_t)a.zero_rows;
        for (int r = threadIdx.x; r < a.zero_rows; r += kFewThreads) keys[r] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kFewThreads) {
            const uint32_t k = key_at(t, i);
            if (k - v0 < (uint32_t)a.zero_rows) keys[k - v0] = 1;
        }
        __syncthreads();
        zero_rows<TG, kFewThreads>(a, v0, t.vocab, [&](uint32_t r) { return keys[r] != 0; });
        return;
    }
    for (int i = threadIdx.x; i < n; i += kFewThreads) keys[i] = key_at(t, i);
    __syncthreads();
    const Window w = window_at(col, a.dim);
    const int mine = blockIdx.x * kFewWaves + wave;
    const uint32_t key = mine < n ? (uint32_t)uniform((int)keys[mine]) : none;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // positions of `k` within [from, to) into this wave's list, in order
    auto gather = [&](uint32_t k, int from, int to) {
        int have = 0;
        for (int j = from; j < to; j += 64) {
            const bool hit = j + lane < to && keys[j + lane] == k;
            const uint64_t m = __ballot(hit);
            if (hit) list[wave][have + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)(j + lane);
            have += __popcll(m);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        return have;
    };
    auto sum = [&](int have) {
        for (int j0 = 0; j0 < have; j0 += kFewBatch) {
            // places behind the end repeat the last one: their rows are not used
            const int here = list[wave][min(j0 + (lane & (kFewBatch - 1)), have - 1)];
            Raw8<TD> raw[kFewBatch];
#pragma unroll
            for (int j = 0; j < kFewBatch; ++j)
                raw[j] = fetch_row<TD, NARROW>(a, __builtin_amdgcn_readlane(here, j), w);
#pragma unroll
            for (int j = 0; j < kFewBatch; ++j)
                if (j0 + j < have)
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[c] += element<TD>(raw[j], c);
        }
    };
    // the first of its token?  how many are there?
    int count = 0;
    if (key != none) {
        bool first = true;
        for (int j = 0; j < mine && first; j += 64) first = __ballot(j + lane < mine && keys[j + lane] == key) == 0;
        if (first)
            for (int j = mine; j < n; j += 64) count += __popcll(__ballot(j + lane < n && keys[j + lane] == key));
    }
    if (count > 0 && count <= kEmbedLong) {
        sum(gather(key, mine, n));
        write_row<TG>(a, key, w.col, w.skip, w.n, acc);
    }
    if (lane == 0) longs[wave] = count > kEmbedLong ? key : none;
    __syncthreads();
    for (int other = 0; other < kFewWaves; ++other) {
        const uint32_t k = (uint32_t)uniform((int)longs[other]);
        if (k == none) continue;
        const int share = (n + kFewThreads - 1) / kFewThreads * 64;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = 0.0f;
        sum(gather(k, min(n, wave * share), min(n, (wave + 1) * share)));
        *reinterpret_cast<v4f*>(&part[wave][lane * 8]) = v4f{acc[0], acc[1], acc[2], acc[3]};
        *reinterpret_cast<v4f*>(&part[wave][lane * 8 + 4]) = v4f{acc[4], acc[5], acc[6], acc[7]};
        __syncthreads();
        if (wave == 0) {
            for (int u = 1; u < kFewWaves; ++u)
#pragma unroll
                for (int c = 0; c < 8; ++c) acc[c] += part[u][lane * 8 + c];
            write_row<TG>(a, k, w.col, w.skip, w.n, acc);
        }
        __syncthreads();
    }
}

int last_error() { return (int)hipGetLastError(); }

template <int TT>
void lookup_to(const EmbedLookup& a, int out, dim3 grid, hipStream_t s) {
    if (out == ZERO_F32) embed_lookup_kernel<TT, ZERO_F32><<<grid, kThreads, 0, s>>>(a);
    else if (out == ZERO_F16) embed_lookup_kernel<TT, ZERO_F16><<<grid, kThreads, 0, s>>>(a);
    else embed_lookup_kernel<TT, ZERO_BF16><<<grid, kThreads, 0, s>>>(a);
}

template <int TD, int TG>
void sum_of(const EmbedSum& a, dim3 grid, hipStream_t s) {
    if (a.dim >= 8) embed_sum_kernel<TD, TG, false><<<grid, kThreads, 0, s>>>(a);
    else embed_sum_kernel<TD, TG, true><<<grid, kThreads, 0, s>>>(a);
}
template <int TD>
void sum_to(const EmbedSum& a, int grad, dim3 grid, hipStream_t s) {
    if (grad == ZERO_F32) sum_of<TD, ZERO_F32>(a, grid, s);
    else if (grad == ZERO_F16) sum_of<TD, ZERO_F16>(a, grid, s);
    else sum_of<TD, ZERO_BF16>(a, grid, s);
}

template <int TD, int TG>
void few_of(const EmbedSort& t, const EmbedSum& a, dim3 grid, hipStream_t s) {
    if (a.dim >= 8) embed_few_kernel<TD, TG, false><<<grid, kFewThreads, 0, s>>>(t, a);
    else embed_few_kernel<TD, TG, true><<<grid, kFewThreads, 0, s>>>(t, a);
}
template <int TD>
void few_to(const EmbedSort& t, const EmbedSum& a, int grad, dim3 grid, hipStream_t s) {
    if (grad == ZERO_F32) few_of<TD, ZERO_F32>(t, a, grid, s);
    else if (grad == ZERO_F16) few_of<TD, ZERO_F16>(t, a, grid, s);
    else few_of<TD, ZERO_BF16>(t, a, grid, s);
}

}  // namespace

int launch_embed_lookup(const EmbedLookupLaunch& l, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t per_row = (l.dim + 7) / 8;
    // groups are counted in 31 bits: more tokens than that take several launches
    const int64_t most = ((int64_t)1 << 30) / per_row;
    EmbedLookup a = l.args;
    a.dim = l.dim;
    a.per_row = make_div((uint32_t)per_row);
    // Large outputs go past the caches, but for fp32 rows of whole 16 bytes from a table
    // of 16 bits: cached and past the caches, us, 16384 x 4096 74, 88, 65536 x 2048 143,
    // 193; x 4095 104, 91; from an fp32 table 65536 x 2048 184, 166; INT8 to fp32 85, 58.
    const bool cached = l.out_dtype == ZERO_F32 && (l.table_dtype == ZERO_F16 || l.table_dtype == ZERO_BF16) &&
                        a.dim % 4 == 0 && a.out_ld % 4 == 0;
    a.stream = !cached && streams(l.n_tokens * l.dim * (l.out_dtype == ZERO_F32 ? 4 : 2));
    for (int64_t t = 0; t < l.n_tokens; t += most) {
        const int64_t n = l.n_tokens - t < most ? l.n_tokens - t : most;
        a.tokens = static_cast<const char*>(l.args.tokens) + t * (a.wide ? 8 : 4);
        a.out = static_cast<char*>(l.args.out) + t * a.out_ld * (l.out_dtype == ZERO_F32 ? 4 : 2);
        a.groups = (uint32_t)(n * per_row);
        const dim3 grid((a.groups + kThreads - 1) / kThreads);
        if (l.table_dtype == kEmbedInt8) lookup_to<kEmbedInt8>(a, l.out_dtype, grid, s);
        else if (l.table_dtype == ZERO_F32) lookup_to<ZERO_F32>(a, l.out_dtype, grid, s);
        else if (l.table_dtype == ZERO_F16) lookup_to<ZERO_F16>(a, l.out_dtype, grid, s);
        else lookup_to<ZERO_BF16>(a, l.out_dtype, grid, s);
        if (const int e = last_error()) return e;
    }
    return 0;
}

int launch_embed_grad(const EmbedGradLaunch& l, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    EmbedSort a = l.sort;
    const int64_t row_bytes = l.sum.dim * (l.grad_dtype == ZERO_F32 ? 4 : 2);
    EmbedSum b = l.sum;
    const int64_t chunks = (row_bytes + 15) / 16;
    b.row_chunks = make_div((uint32_t)chunks);
    // Past the caches dy stays in them: 16384 x 4096 into 32000 bf16 rows 90 us, cached 94.
    // Few tokens have little dy: 256 x 4096 into the same 40 cached, 56 past the caches.
    // Of an accumulated gradient only the rows that tokens name are written.
    b.stream = !embed_few(a.n_tokens, b.dim) && streams((b.accumulate ? (a.n_tokens < a.vocab ? a.n_tokens : a.vocab) : a.vocab) * row_bytes);
    if (embed_few(a.n_tokens, b.dim)) {
        const int64_t rows = l.sum.accumulate ? 0 : a.vocab, each = (rows + kFewBlocks - 1) / kFewBlocks;
        // their marks lie where the tokens' rows do otherwise
        b.zero_rows = (int32_t)(each < kFewRows ? kFewRows : each > kEmbedFew ? kEmbedFew : each);
        if (b.zero_rows > (1 << 29) / chunks) b.zero_rows = (int32_t)((1 << 29) / chunks);
        const dim3 grid((uint32_t)((a.n_tokens + kFewWaves - 1) / kFewWaves + (rows + b.zero_rows - 1) / b.zero_rows),
                        (uint32_t)((b.dim + kChunk - 1) / kChunk));
        if (l.dy_dtype == ZERO_F32) few_to<ZERO_F32>(a, b, l.grad_dtype, grid, s);
        else if (l.dy_dtype == ZERO_F16) few_to<ZERO_F16>(a, b, l.grad_dtype, grid, s);
        else few_to<ZERO_BF16>(a, b, l.grad_dtype, grid, s);
        return last_error();
    }
    char* ws = static_cast<char*>(l.workspace);
    const EmbedWorkspace w = embed_workspace(a.n_tokens, a.vocab, l.sum.dim);
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + w.keys[0]), reinterpret_cast<uint32_t*>(ws + w.keys[1])};
    int32_t* places[2] = {reinterpret_cast<int32_t*>(ws + w.places[0]), reinterpret_cast<int32_t*>(ws + w.places[1])};
    a.flags = l.sum.accumulate ? nullptr : reinterpret_cast<uint32_t*>(ws + w.flags);
    a.flag_words = (a.vocab + 3) / 4;
    a.hist = reinterpret_cast<uint32_t*>(ws + w.hist);
    int bits = 1;
    while ((a.vocab >> bits) != 0) ++bits;                 // keys are 0 .. vocab
    a.passes = (bits + 7) / 8;
    a.digit_bits = (bits + a.passes - 1) / a.passes;
    a.blocks = (int32_t)((a.n_tokens + kEmbedSortTile - 1) / kEmbedSortTile);
    a.scanned = a.blocks > kEmbedScanBlocks;
    // each launch of the sort writes so many bytes of zeros beside its work
    const int64_t total = l.sum.accumulate ? 0 : a.vocab * row_bytes;
    a.grad = static_cast<char*>(l.sum.grad);
    a.stream = b.stream;
    const auto grid = [&]() {
        a.zero_first = a.zero_last;
        a.zero_last = total - a.zero_first < kEmbedZeroBytes ? total : a.zero_first + kEmbedZeroBytes;
        return dim3((uint32_t)(a.blocks + (a.zero_last - a.zero_first + kZeroBlock - 1) / kZeroBlock));
    };
    int at = 0;
    for (a.pass = 0; a.pass < a.passes; ++a.pass) {
        a.keys_in = keys[at];
        a.places_in = places[at];
        at ^= 1;
        a.keys_out = keys[at];
        a.places_out = places[at];
        dim3 blocks = grid();
        embed_hist_kernel<<<blocks, kThreads, 0, s>>>(a);
        if (const int e = last_error()) return e;
        if (a.scanned) {
            embed_scan_kernel<<<kBins, kThreads, 0, s>>>(a);
            if (const int e = last_error()) return e;
        }
        blocks = grid();
        embed_scatter_kernel<<<blocks, kThreads, 0, s>>>(a);
        if (const int e = last_error()) return e;
    }
    b.keys = keys[at];
    b.places = places[at];
    b.flags = a.flags;
    b.n_tokens = a.n_tokens;
    b.vocab = a.vocab;
    b.partials = reinterpret_cast<float*>(ws + w.partials);
    b.tile = w.tile;
    b.tiles = w.tiles;
    b.pitch = w.pitch;
    b.chunks = (b.dim + kChunk - 1) / kChunk;
    b.sum_blocks = b.tiles * b.chunks;
    // rows that are zero already need no more of it; one that is so in part does
    b.zero_from = b.accumulate ? b.vocab : a.zero_last / row_bytes;
    const int64_t each = kZeroRowsBytes / row_bytes;
    b.zero_rows = (int32_t)(each < 4 ? 4 : each > 64 ? 64 : each);
    const dim3 sums((uint32_t)(b.sum_blocks + (b.vocab - b.zero_from + b.zero_rows - 1) / b.zero_rows));
    if (l.dy_dtype == ZERO_F32) sum_to<ZERO_F32>(b, l.grad_dtype, sums, s);
    else if (l.dy_dtype == ZERO_F16) sum_to<ZERO_F16>(b, l.grad_dtype, sums, s);
    else sum_to<ZERO_BF16>(b, l.grad_dtype, sums, s);
    if (const int e = last_error()) return e;
    if (b.tiles > 1) {
        const dim3 joins((uint32_t)(b.tiles - 1), (uint32_t)b.chunks);
        if (l.grad_dtype == ZERO_F32) embed_join_kernel<ZERO_F32><<<joins, kThreads, 0, s>>>(b);
        else if (l.grad_dtype == ZERO_F16) embed_join_kernel<ZERO_F16><<<joins, kThreads, 0, s>>>(b);
        else embed_join_kernel<ZERO_BF16><<<joins, kThreads, 0, s>>>(b);
        if (const int e = last_error()) return e;
    }
    return 0;
}

}  // namespace zf
