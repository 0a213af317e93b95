// zeroflat_wgrad.hip -- gfx950 (MI355X, CDNA4, wave64) kernels of a linear
// layer's weight gradient from the 8-bit checkpoint of its input:
//   weight_grad_kernel  grad[o][i] = sum over rows t of dy[t][o] * x[t][i] on the
//                       matrix cores, a tile of grad per block
//   weight_join_kernel  the partial sums of a product split over its rows
//
// Both operands lie with the summed index outermost, while a lane of a matrix
// instruction wants eight consecutive values of it: tiles go to LDS as they lie
// in memory and are read back by the transposing LDS load.  The codes are
// restored on the way into LDS, once per block: code * 2^k is exact in bf16, so
// the products are exact in fp32 and only their sums round.
//
// The large tile, 256 x 256 by eight waves, needs every register: a wave's 128 sums,
// the operands of one step, which give way to the next one's row by row, and two steps
// of loads.  4096 x 4096 over 16384 rows take 432 us, 1.27 PFLOP/s in bf16 (a library
// product of two 8192 x 8192 matrices 1.29, of these two operands in bf16 0.93).  Tried
// and not kept: both halves of a step's operands held twice (spills; 720 us), four waves
// of 128 x 128 (the sums move between register files; spills), loads one step ahead
// (496 us), an exclusive-or order of LDS in place of the pad (a register per fragment),
// four buffers and a barrier for every second step (489 us without a spill in the loop).
#include "zf_vec.h"

namespace zf {
namespace {

typedef signed char v4c __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

template <int DT>
__device__ __forceinline__ v4f mfma(v8s a, v8s b, v4f c) {
    if constexpr (DT == ZERO_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// A row of a tile in LDS is T 16-bit elements and 16 more: the transposing load's
// lanes read 32 bytes of rows in turn, eight of which then fill the banks once, and
// every address of a lane is one number and a constant.
constexpr int kPad = 16;

__device__ __forceinline__ float scale_of(uint32_t exponent) {
    return exponent == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((exponent - 6u) << 23);
}
// Four codes to 16-bit values.
template <int DT>
__device__ __forceinline__ v2u restore4(uint32_t codes, float s) {
    const v4c c = __builtin_bit_cast(v4c, codes);
    v2u out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float a = (float)c[2 * h] * s, b = (float)c[2 * h + 1] * s;
        if constexpr (DT == ZERO_BF16)     // exact: the low halves are zero
            out[h] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        else
            out[h] = (uint32_t)from_f32<ZERO_F16>(a) | (uint32_t)from_f32<ZERO_F16>(b) << 16;
    }
    return out;
}

// Four consecutive elements at any element offset, the first n of which exist.
template <int DT>
__device__ __forceinline__ v4f read4(const void* base, int64_t at, int n) {
    const auto* p = static_cast<const typename Elem<DT>::type*>(base) + at;
    v4f x = {0, 0, 0, 0};
    if (n >= 4) {
        if constexpr (DT == ZERO_F32) {
            x = *reinterpret_cast<const v4f_any*>(p);
        } else {
            const v2u w = *reinterpret_cast<const v2u_any*>(p);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = to_f32<DT>((uint16_t)(w[k / 2] >> (16 * (k & 1))));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) x[k] = to_f32<DT>(p[k]);
    }
    return x;
}
template <int DT>
__device__ __forceinline__ void write4(void* base, int64_t at, int n, v4f x) {
    auto* p = static_cast<typename Elem<DT>::type*>(base) + at;
    if (n >= 4) {
        if constexpr (DT == ZERO_F32) {
            *reinterpret_cast<v4f_any*>(p) = x;
        } else {
            v2u w;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w[h] = (uint32_t)from_f32<DT>(x[2 * h]) | (uint32_t)from_f32<DT>(x[2 * h + 1]) << 16;
            *reinterpret_cast<v2u_any*>(p) = w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
            if (k < n) p[k] = from_f32<DT>(x[k]);
    }
}
// The sum into the gradient: one rounding to its type, after the addition.
template <int DT>
__device__ __forceinline__ void finish4_as(const WeightGrad& a, int64_t at, int n, v4f x) {
    if (a.accumulate) {
        const v4f old = read4<DT>(a.grad, at, n);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] += old[k];
    }
    write4<DT>(a.grad, at, n, x);
}
__device__ __forceinline__ void finish4(const WeightGrad& a, int64_t at, int n, v4f x) {
    if (a.grad_dtype == ZERO_F32) finish4_as<ZERO_F32>(a, at, n, x);
    else if (a.grad_dtype == ZERO_F16) finish4_as<ZERO_F16>(a, at, n, x);
    else finish4_as<ZERO_BF16>(a, at, n, x);
}

// What block b does.  The first blocks take whole tiles, the ones behind them
// shares of the rows of the tiles that are left.  Blocks go to the eight dies in
// turn: each die gets a run of tiles, in bands of four, so that the tiles it has
// at a time share their strips of dy and x in its cache.
struct Unit {
    uint32_t to, ti, split, part;
    bool shared;
};
__device__ __forceinline__ Unit unit_of(const WeightGrad& a, uint32_t b) {
    Unit u;
    const uint32_t cut = (uint32_t)a.whole_tiles, rest = (uint32_t)a.tiles - cut;
    u.shared = b >= cut;
    u.part = b - cut;
    u.split = u.shared ? u.part / rest : 0;
    const uint32_t nth = u.shared ? u.part - u.split * rest : b, in_run = u.shared ? rest : cut;
    const uint32_t die = nth % 8, tile = (u.shared ? cut : 0) + die * (in_run / 8) + min(die, in_run % 8) + nth / 8;
    const uint32_t wide = (uint32_t)a.tiles_i, band = tile / (4 * wide), in_band = tile - band * 4 * wide;
    const uint32_t high = min(4u, (uint32_t)a.tiles_o - band * 4);
    u.to = band * 4 + in_band % high;
    u.ti = in_band / high;
    return u;
}

// A block's tile is TO outputs o by TI inputs i, its waves WO by WI of them; a step is
// DEPTH rows t, 32 for every matrix instruction.
template <int TO, int TI, int WO, int WI, int DEPTH>
struct Tile {
    static constexpr int threads = WO * WI * 64;
    static constexpr int fo = TO / WO / 16, fi = TI / WI / 16;      // 16 x 16 fragments of a wave
    static constexpr int y_loads = DEPTH * TO / 8 / threads;       // 16 bytes each
    static constexpr int x_loads = DEPTH * TI / 16 / threads;
    static_assert(y_loads * 8 * threads == DEPTH * TO && x_loads * 16 * threads == DEPTH * TI, "whole loads");
};

template <int DT, int TO, int TI, int WO, int WI, int DEPTH, int SETS>
__global__ __launch_bounds__(WO * WI * 64, 2) void weight_grad_kernel(WeightGrad a) {
    using S = Tile<TO, TI, WO, WI, DEPTH>;
    constexpr int ly = TO + kPad, lx = TI + kPad;
    __shared__ __attribute__((aligned(16))) uint16_t ysh[2 * DEPTH * ly];
    __shared__ __attribute__((aligned(16))) uint16_t xsh[2 * DEPTH * lx];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const Unit u = unit_of(a, blockIdx.x);
    const int64_t o0 = (int64_t)u.to * TO, i0 = (int64_t)u.ti * TI;
    const bool shared = u.shared;
    const int64_t t0 = shared ? u.split * a.share : 0, t1 = shared ? min(a.rows, t0 + a.share) : a.rows;
    const int steps = (int)((t1 - t0 + DEPTH - 1) / DEPTH);
    // Steps whose loads need no test.  Columns beyond the matrix are read from
    // inside it (their results are not written), but for a last group of fewer
    // than eight outputs, which runs into the next row: there has to be one.  A
    // thread's rows are within 32 bits of a step's first.
    const bool over = a.outs % 8 != 0;
    const int whole = a.outs < 8 || (over && a.dy_ld < a.outs) || a.dy_ld > (int64_t)1 << 25 ? 0
        : (int)((min(t1, a.rows - (over ? 1 : 0)) - t0) / DEPTH);

    // This thread's part of a step: groups of eight outputs and of sixteen codes.
    constexpr int ywide = TO / 8, xwide = TI / 16;             // in a row
    constexpr int yrows = S::threads / ywide, xrows = S::threads / xwide;   // rows apart
    static_assert(yrows * ywide == S::threads && xrows * xwide == S::threads, "whole rows per load");
    const int ycol = tid % ywide * 8, yk = tid / ywide;
    const int xcol = tid % xwide * 16, xk = tid / xwide;
    const int64_t o = min(o0 + ycol, (a.outs - 1) / 8 * 8), i = min(i0 + xcol, a.pitch - 16);
    // a step's first row, the same for the whole block, and this thread's place in bytes
    const char* yp = static_cast<const char*>(a.dy) + t0 * a.dy_ld * 2;
    const char* xp = reinterpret_cast<const char*>(a.codes) + t0 * a.pitch;
    const char* ep = reinterpret_cast<const char*>(a.exponents) + t0 * (a.pitch / 32);
    const uint32_t yat = (uint32_t)(yk * a.dy_ld + o) * 2, xat = (uint32_t)(xk * a.pitch + i);
    const uint32_t eat = (uint32_t)(xk * (a.pitch / 32) + i / 32);
    const int64_t ystep = yrows * a.dy_ld * 2, xstep = xrows * a.pitch;

    // SETS steps' loads on their way
    static_assert(SETS % 2 == 0, "a set goes to one buffer");
    v4u yreg[SETS][S::y_loads], xreg[SETS][S::x_loads];
    uint32_t ereg[SETS][S::x_loads];
    auto fetch_y = [&](int set, int j) { yreg[set][j] = *reinterpret_cast<const v4u_any*>(yp + j * ystep + yat); };
    auto fetch_x = [&](int set, int j) {
        xreg[set][j] = *reinterpret_cast<const v4u*>(xp + j * xstep + xat);
        ereg[set][j] = *reinterpret_cast<const uint8_t*>(ep + j * (xstep / 32) + eat);
    };
    auto advance = [&]() {
        yp += DEPTH * a.dy_ld * 2;
        xp += DEPTH * a.pitch;
        ep += DEPTH * (a.pitch / 32);
    };
    auto fetch = [&](int set, int n) {         // step n, zeros beyond the rows
        if (n >= steps) return;
        // its addresses are made anew from the thread's number: kept over the main
        // loop they would take the registers that its loads need
        int id = tid;
        asm volatile("" : "+v"(id));
        const int yk = id / ywide, xk = id / xwide;
        const int64_t o = min(o0 + id % ywide * 8, (a.outs - 1) / 8 * 8), i = min(i0 + id % xwide * 16, a.pitch - 16);
        const int64_t t = t0 + (int64_t)n * DEPTH;
#pragma unroll
        for (int j = 0; j < S::y_loads; ++j) {
            const int64_t row = t + yk + j * yrows;
            yreg[set][j] = v4u{0, 0, 0, 0};
            if (row < t1) {
                const uint16_t* p = static_cast<const uint16_t*>(a.dy) + row * a.dy_ld + o;
                if (o + 8 <= a.outs) {
                    yreg[set][j] = *reinterpret_cast<const v4u_any*>(p);
                } else {
#pragma unroll
                    for (int q = 0; q < 7; ++q)
                        if (o + q < a.outs) yreg[set][j][q / 2] |= (uint32_t)p[q] << (16 * (q & 1));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < S::x_loads; ++j) {
            const int64_t row = t + xk + j * xrows;
            xreg[set][j] = v4u{0, 0, 0, 0};
            ereg[set][j] = 7;
            if (row < t1) {
                xreg[set][j] = *reinterpret_cast<const v4u*>(a.codes + row * a.pitch + i);
                ereg[set][j] = a.exponents[row * (a.pitch / 32) + i / 32];
            }
        }
    };
    // set k goes to buffer k % 2
    auto stage_y = [&](int set, int j) {
        *reinterpret_cast<v4u*>(&ysh[(set % 2 * DEPTH + yk + j * yrows) * ly + ycol]) = yreg[set][j];
    };
    v4u half;
    auto stage_x = [&](int set, int w) {       // word w % 4 of load w / 4
        const v2u r = restore4<DT>(xreg[set][w / 4][w % 4], scale_of(ereg[set][w / 4]));
        half[2 * (w & 1)] = r[0];
        half[2 * (w & 1) + 1] = r[1];
        if (w & 1)
            *reinterpret_cast<v4u*>(&xsh[(set % 2 * DEPTH + xk + w / 4 * xrows) * lx + xcol + (w & 2) * 4]) = half;
    };
    auto stage = [&](int set) {
#pragma unroll
        for (int j = 0; j < S::y_loads; ++j) stage_y(set, j);
#pragma unroll
        for (int w = 0; w < 4 * S::x_loads; ++w) stage_x(set, w);
    };

    v4f acc[S::fo][S::fi];
#pragma unroll
    for (int o = 0; o < S::fo; ++o)
#pragma unroll
        for (int i = 0; i < S::fi; ++i) acc[o][i] = v4f{0, 0, 0, 0};
    const int wo = wave / WI * S::fo, wi = wave % WI * S::fi;
    // This lane's row of a transposing load.  The sum's order is free as long as both
    // operands have the same one: a lane's eight values are of rows 4g to 4g + 3 and
    // 16 more, so that the lanes of a load read sixteen rows in turn (with eight rows in
    // turn, each second group of four left out, two of them met in every bank: 449 us
    // for the head's 432, and LDS busy with conflicts for 27% of the time, now 7).
    const int krow = lane / 4;
    const int kcol = lane % 4 * 4;
    constexpr int parts = DEPTH / 32;
    v8s x[parts][S::fi], y[parts][S::fo];       // a step's operands
    auto frag = [&](const uint16_t* p, int row) {
        const v4s u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
        const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 16 * row));
        return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    const uint16_t* xread = xsh + krow * lx + kcol + wi * 16;
    const uint16_t* yread = ysh + krow * ly + kcol + wo * 16;
    auto xfrag = [&](int buf, int part, int i) { return frag(xread + (buf * DEPTH + part * 32) * lx + i * 16, lx); };
    auto yfrag = [&](int buf, int part, int o) { return frag(yread + (buf * DEPTH + part * 32) * ly + o * 16, ly); };
    // Multiplies the step whose operands are held; row by row they give way to those of
    // the next one, in the other buffer, and `work` gets its turns beside them.
    constexpr int turns = parts * S::fo;
    auto multiply = [&](int buf, bool more, auto work) {
#pragma unroll
        for (int p = 0; p < parts; ++p)
#pragma unroll
            for (int o = 0; o < S::fo; ++o) {
#pragma unroll
                for (int i = 0; i < S::fi; ++i) {
                    acc[o][i] = mfma<DT>(x[p][i], y[p][o], acc[o][i]);
                    if (more && o == S::fo - 1) x[p][i] = xfrag(1 - buf, p, i);
                }
                if (more) y[p][o] = yfrag(1 - buf, p, o);
                work(p * S::fo + o);
                __builtin_amdgcn_sched_barrier(0);
            }
    };

    // Step s multiplies what was read from buffer s % 2 during step s - 1, reads step
    // s + 1 from the other buffer, writes step s + 2 over its own and issues the loads
    // of step s + 2 + SETS.  Step n's loads are in set n % SETS.
    if (steps > 0) {
        fetch(0, 0);
        fetch(1, 1);
        stage(0);
        if (steps > 1) stage(1);
#pragma unroll
        for (int n = 2; n < 2 + SETS; ++n) fetch(n % SETS, n);
        __syncthreads();
#pragma unroll
        for (int p = 0; p < parts; ++p) {
#pragma unroll
            for (int i = 0; i < S::fi; ++i) x[p][i] = xfrag(0, p, i);
#pragma unroll
            for (int o = 0; o < S::fo; ++o) y[p][o] = yfrag(0, p, o);
        }
        __syncthreads();
    }
    int s = 0;
    yp += (2 + SETS) * DEPTH * a.dy_ld * 2;
    xp += (2 + SETS) * DEPTH * a.pitch;
    ep += (2 + SETS) * DEPTH * (a.pitch / 32);
    for (; s + 2 * SETS + 1 < whole; s += SETS) {
#pragma unroll
        for (int k = 0; k < SETS; ++k) {
            const int set = (k + 2) % SETS;
            multiply(k % 2, true, [&](int turn) {
#pragma unroll
                for (int j = turn * S::y_loads / turns; j < (turn + 1) * S::y_loads / turns; ++j) {
                    stage_y(set, j);
                    fetch_y(set, j);
                }
#pragma unroll
                for (int w = turn * 4 * S::x_loads / turns; w < (turn + 1) * 4 * S::x_loads / turns; ++w) {
                    stage_x(set, w);
                    if (w % 4 == 3) fetch_x(set, w / 4);
                }
            });
            advance();
            __syncthreads();
        }
    }
    for (; s < steps; s += SETS) {
#pragma unroll
        for (int k = 0; k < SETS; ++k) {
            if (s + k < steps) {
                const int set = (k + 2) % SETS;
                if (s + k + 2 < steps) stage(set);
                fetch(set, s + k + 2 + SETS);
                multiply(k % 2, s + k + 1 < steps, [](int) {});
                __syncthreads();
            }
        }
    }

    // a lane has four consecutive inputs i of one output o
#pragma unroll
    for (int o = 0; o < S::fo; ++o) {
        const int64_t row = o0 + (wo + o) * 16 + lane % 16;
        if (row >= a.outs) continue;
#pragma unroll
        for (int i = 0; i < S::fi; ++i) {
            const int64_t col = i0 + (wi + i) * 16 + lane / 16 * 4;
            const int n = (int)min((int64_t)4, a.cols - col);
            if (n <= 0) continue;
            if (shared) {
                // by unit, wave, fragment and lane: whole lines
                float* p = a.partials + (int64_t)u.part * (TO * TI);
                *reinterpret_cast<v4f*>(p + (((wave * S::fo + o) * S::fi + i) * 64 + lane) * 4) = acc[o][i];
            } else {
                finish4(a, row * a.cols + col, n, acc[o][i]);
            }
        }
    }
}

// The shares' sums of a tile added in order: four elements per thread.
template <int TO, int TI, int WO, int WI, int DEPTH>
__global__ __launch_bounds__(256) void weight_join_kernel(WeightGrad a) {
    using S = Tile<TO, TI, WO, WI, DEPTH>;
    constexpr uint32_t blocks = TO * TI / 1024;
    const uint32_t rest = (uint32_t)(a.tiles - a.whole_tiles), nth = blockIdx.x / blocks;
    const Unit u = unit_of(a, (uint32_t)a.whole_tiles + nth);
    const int q = (int)(blockIdx.x % blocks) * 256 + threadIdx.x, lane = q & 63, frag = q >> 6;
    const int i = frag % S::fi, o = frag / S::fi % S::fo, wave = frag / (S::fi * S::fo);
    const int64_t row = (int64_t)u.to * TO + (wave / WI * S::fo + o) * 16 + lane % 16;
    const int64_t col = (int64_t)u.ti * TI + (wave % WI * S::fi + i) * 16 + lane / 16 * 4;
    const int n = (int)min((int64_t)4, a.cols - col);
    if (row >= a.outs || n <= 0) return;
    const float* p = a.partials + (int64_t)nth * (TO * TI) + q * 4;
    v4f sum = *reinterpret_cast<const v4f*>(p);
#pragma unroll 4
    for (int s = 1; s < a.splits; ++s) {
        const v4f x = *reinterpret_cast<const v4f*>(p + (int64_t)s * rest * (TO * TI));
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] += x[k];
    }
    finish4(a, row * a.cols + col, n, sum);
}

template <int DT, int TO, int TI, int WO, int WI, int DEPTH, int SETS>
int launch_tile(const WeightGrad& a, hipStream_t s) {
    const int64_t rest = a.tiles - a.whole_tiles;
    weight_grad_kernel<DT, TO, TI, WO, WI, DEPTH, SETS><<<(uint32_t)(a.whole_tiles + rest * a.splits), WO * WI * 64, 0, s>>>(a);
    if (const int e = (int)hipGetLastError()) return e;
    if (rest) weight_join_kernel<TO, TI, WO, WI, DEPTH><<<(uint32_t)(rest * (TO * TI / 1024)), 256, 0, s>>>(a);
    return (int)hipGetLastError();
}
template <int DT>
int launch_dt(const WeightGrad& a, hipStream_t s) {
    if (a.tile == 256) return launch_tile<DT, 256, 256, 2, 4, 32, 2>(a, s);
    if (a.tile == 128) return launch_tile<DT, 128, 128, 2, 2, 64, 2>(a, s);
    return launch_tile<DT, 64, 64, 2, 2, 64, 2>(a, s);
}

}  // namespace

// The tile and the split: the least of the times that the measured parts add up to.
// A tile's blocks fill `slots` places of the chip; whole rounds of tiles are summed
// by a block each, and the tiles left over, which would leave places empty, may be
// shared by blocks, whose sums (fp32) cost their writing and reading.  In ns: 32 rows
// with up to `free` blocks at once and with every place taken, a block's beginning and
// end, a share's traffic, the second launch.  Large tiles move fewer bytes per product,
// small ones spread small gradients over the chip.  Measured, the best split of each,
// us: 512 x 1024 over 512 rows 9.2, 13.2, 17.0 with tiles of 64, 128, 256; 1024 x 1024
// over 2048 rows 20.9, 21.8, 27.0; over 8192 rows 47.9, 34.8, 41.3; 2048 x 2048 over 2048
// rows 54.6, 33.5, 43.2; 4096 x 4096 over 2048 rows 96, 67 with 128, 256; 4099 x 4001
// over 16384 rows 732, 488 (unsplit 906, 825).
void plan_weight_grad(WeightGrad& a) {
    struct Kind {
        int64_t tile, slots, free, step, step_full, ends, part;
    };
    static const Kind kinds[] = {{256, 256, 0, 740, 880, 6000, 86},
                                 {128, 512, 256, 380, 660, 6000, 22},
                                 {64, 1024, 256, 235, 775, 5500, 6}};
    static const int64_t splits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96};
    const int64_t steps = (a.rows + 31) / 32;
    int64_t best = INT64_MAX;
    for (const Kind& k : kinds) {
        const int64_t to = (a.outs + k.tile - 1) / k.tile, ti = (a.cols + k.tile - 1) / k.tile, tiles = to * ti;
        const auto round = [&](int64_t n, int64_t units) {     // n steps of `units` blocks at once
            const int64_t more = units > k.free ? units - k.free : 0;
            return n * (k.step + (k.step_full - k.step) * more / (k.slots - k.free)) + k.ends;
        };
        for (const int64_t s : splits) {
            if (s > 1 && s * 2 > steps) break;
            const int64_t whole = s == 1 ? tiles : tiles / k.slots * k.slots, rest = tiles - whole;
            if (s > 1 && rest == 0) break;
            const int64_t units = rest * s, share = (steps + s - 1) / s;
            int64_t time = whole / k.slots * round(steps, k.slots);
            if (whole % k.slots) time += round(steps, whole % k.slots);
            if (units) {
                time += units / k.slots * round(share, k.slots) + units * k.part + 3000;
                if (units % k.slots) time += round(share, units % k.slots);
            }
            if (time >= best) continue;
            best = time;
            a.tile = (int32_t)k.tile;
            a.tiles_o = to;
            a.tiles_i = ti;
            a.tiles = tiles;
            a.whole_tiles = whole;
            a.share = share * 32;
            a.splits = s == 1 ? 1 : (int32_t)((a.rows + a.share - 1) / a.share);
        }
    }
}

int launch_weight_grad(const WeightGrad& a, int dtype, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return dtype == ZERO_BF16 ? launch_dt<ZERO_BF16>(a, s) : launch_dt<ZERO_F16>(a, s);
}

}  // namespace zf
