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
#include "zf_vec.h"

namespace zf {
namespace {

constexpr int kDepth = 64;                 // rows t of one step

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

// A row of a tile in LDS is T 16-bit elements in chunks of 16, each at its place
// xor a number of the row: the transposing load's sixteen lanes read one chunk
// of four rows, which then lie in different banks.
template <int T>
__device__ __forceinline__ int swizzle(int k) {
    return ((k & 3) | ((k >> 3) & 1) << 2) & (T / 16 - 1);
}

// Sixteen codes with one exponent to 16-bit values.
template <int DT>
__device__ __forceinline__ void restore16(v4u codes, uint32_t exponent, v4u& lo, v4u& hi) {
    const float s = exponent == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((exponent - 6u) << 23);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t word = codes[w];
        const v4c c = __builtin_bit_cast(v4c, word);
        uint32_t out[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = (float)c[2 * h] * s, b = (float)c[2 * h + 1] * s;
            if constexpr (DT == ZERO_BF16)     // exact: the low halves are zero
                out[h] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
            else
                out[h] = (uint32_t)from_f32<ZERO_F16>(a) | (uint32_t)from_f32<ZERO_F16>(b) << 16;
        }
        v4u& to = w < 2 ? lo : hi;
        to[2 * (w & 1)] = out[0];
        to[2 * (w & 1) + 1] = out[1];
    }
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

// A block's tile is TO outputs o by TI inputs i, its waves WO by WI of them.
template <int DT, int TO, int TI, int WO, int WI>
struct Tile {
    static constexpr int threads = WO * WI * 64;
    static constexpr int fo = TO / WO / 16, fi = TI / WI / 16;      // 16 x 16 fragments of a wave
    static constexpr int y_loads = kDepth * TO / 8 / threads;       // 16 bytes each
    static constexpr int x_loads = kDepth * TI / 16 / threads;
    static_assert(y_loads * 8 * threads == kDepth * TO && x_loads * 16 * threads == kDepth * TI, "whole loads");
};

template <int DT, int TO, int TI, int WO, int WI>
__global__ __launch_bounds__(WO * WI * 64) void weight_grad_kernel(WeightGrad a) {
    using S = Tile<DT, TO, TI, WO, WI>;
    __shared__ __attribute__((aligned(16))) uint16_t ysh[2][kDepth * TO];
    __shared__ __attribute__((aligned(16))) uint16_t xsh[2][kDepth * TI];
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int64_t b = blockIdx.x;
    const int64_t split = b / a.tiles, tile = b - split * a.tiles;
    const int64_t to = tile / a.tiles_i, ti = tile - to * a.tiles_i;
    const int64_t o0 = to * TO, i0 = ti * TI;
    const int64_t t0 = split * a.share, t1 = min(a.rows, t0 + a.share);
    const int steps = (int)((t1 - t0 + kDepth - 1) / kDepth);
    // Steps whose loads need no test.  Columns beyond the matrix are read from
    // inside it (their results are not written), but for a last group of fewer
    // than eight outputs, which runs into the next row: there has to be one.
    const bool over = a.outs % 8 != 0;
    const int whole = a.outs < 8 || (over && a.dy_ld < a.outs) ? 0
        : (int)((min(t1, a.rows - (over ? 1 : 0)) - t0) / kDepth);

    // This thread's part of a step: groups of eight outputs and of sixteen codes.
    constexpr int ywide = TO / 8, xwide = TI / 16;             // in a row
    constexpr int yrows = S::threads / ywide, xrows = S::threads / xwide;   // rows apart
    static_assert(yrows * ywide == S::threads && xrows * xwide == S::threads, "whole rows per load");
    const int ycol = tid % ywide * 8, yk = tid / ywide;
    const int xcol = tid % xwide * 16, xk = tid / xwide;
    const int64_t o = min(o0 + ycol, (a.outs - 1) / 8 * 8), i = min(i0 + xcol, a.pitch - 16);
    const uint16_t* yp = static_cast<const uint16_t*>(a.dy) + (t0 + yk) * a.dy_ld + o;
    const int8_t* xp = a.codes + (t0 + xk) * a.pitch + i;
    const uint8_t* ep = a.exponents + (t0 + xk) * (a.pitch / 32) + i / 32;
    const int64_t ystep = yrows * a.dy_ld, xstep = xrows * a.pitch;

    v4u yreg[S::y_loads], xreg[S::x_loads];
    uint32_t ereg[S::x_loads];
    auto fetch = [&]() {                       // of a whole step
#pragma unroll
        for (int j = 0; j < S::y_loads; ++j, yp += ystep) yreg[j] = *reinterpret_cast<const v4u_any*>(yp);
#pragma unroll
        for (int j = 0; j < S::x_loads; ++j, xp += xstep, ep += xstep / 32) {
            xreg[j] = *reinterpret_cast<const v4u*>(xp);
            ereg[j] = *ep;
        }
    };
    auto fetch_some = [&](int step) {          // of any step, zeros beyond the rows
        const int64_t t = t0 + (int64_t)step * kDepth;
#pragma unroll
        for (int j = 0; j < S::y_loads; ++j) {
            const int64_t row = t + yk + j * yrows;
            yreg[j] = v4u{0, 0, 0, 0};
            if (row < t1) {
                const uint16_t* p = static_cast<const uint16_t*>(a.dy) + row * a.dy_ld + o;
                if (o + 8 <= a.outs) {
                    yreg[j] = *reinterpret_cast<const v4u_any*>(p);
                } else {
#pragma unroll
                    for (int q = 0; q < 7; ++q)
                        if (o + q < a.outs) yreg[j][q / 2] |= (uint32_t)p[q] << (16 * (q & 1));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < S::x_loads; ++j) {
            const int64_t row = t + xk + j * xrows;
            xreg[j] = v4u{0, 0, 0, 0};
            ereg[j] = 7;
            if (row < t1) {
                xreg[j] = *reinterpret_cast<const v4u*>(a.codes + row * a.pitch + i);
                ereg[j] = a.exponents[row * (a.pitch / 32) + i / 32];
            }
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int j = 0; j < S::y_loads; ++j) {
            const int k = yk + j * yrows;
            const int at = k * TO + (((ycol >> 4) ^ swizzle<TO>(k)) << 4) + (ycol & 8);
            *reinterpret_cast<v4u*>(&ysh[buf][at]) = yreg[j];
        }
#pragma unroll
        for (int j = 0; j < S::x_loads; ++j) {
            const int k = xk + j * xrows;
            const int at = k * TI + (((xcol >> 4) ^ swizzle<TI>(k)) << 4);
            v4u lo, hi;
            restore16<DT>(xreg[j], ereg[j], lo, hi);
            *reinterpret_cast<v4u*>(&xsh[buf][at]) = lo;
            *reinterpret_cast<v4u*>(&xsh[buf][at + 8]) = hi;
        }
    };

    v4f acc[S::fo][S::fi];
#pragma unroll
    for (int o = 0; o < S::fo; ++o)
#pragma unroll
        for (int i = 0; i < S::fi; ++i) acc[o][i] = v4f{0, 0, 0, 0};
    const int wo = wave / WI * S::fo, wi = wave % WI * S::fi;
    const int krow = 8 * (lane / 16) + lane % 16 / 4;            // this lane's row of a transposing load
    const int kcol = lane % 4 * 4;
    v8s x[S::fi], y[S::fo];
    auto operands = [&](int buf, int half) {
        auto frag = [&](const uint16_t* sh, int T, int chunk) {
            const uint16_t* p = sh + (half + krow) * T + (chunk << 4) + kcol;
            const v4s u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
            const v4s v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * T));
            return __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7);
        };
#pragma unroll
        for (int i = 0; i < S::fi; ++i) x[i] = frag(xsh[buf], TI, (wi + i) ^ swizzle<TI>(krow));
#pragma unroll
        for (int o = 0; o < S::fo; ++o) y[o] = frag(ysh[buf], TO, (wo + o) ^ swizzle<TO>(krow));
    };
    auto multiply = [&]() {
#pragma unroll
        for (int o = 0; o < S::fo; ++o)
#pragma unroll
            for (int i = 0; i < S::fi; ++i) acc[o][i] = mfma<DT>(x[i], y[o], acc[o][i]);
    };

    // While step s is multiplied, the next step's registers go to the other buffer
    // and the loads of the step after that are on their way.
    if (steps > 0) {
        if (whole > 0) fetch();
        else fetch_some(0);
        stage(0);
        if (whole > 1) fetch();
        else if (steps > 1) fetch_some(1);
        __syncthreads();
    }
    int s = 0;
    for (; s + 2 < whole; ++s) {
        operands(s & 1, 0);
        stage((s + 1) & 1);
        fetch();
        __builtin_amdgcn_sched_barrier(0);
        multiply();
        operands(s & 1, 32);
        multiply();
        __syncthreads();
    }
    for (; s < steps; ++s) {
        if (s + 1 < steps) stage((s + 1) & 1);
        if (s + 2 < steps) fetch_some(s + 2);
        operands(s & 1, 0);
        multiply();
        operands(s & 1, 32);
        multiply();
        __syncthreads();
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
            if (a.partials) write4<ZERO_F32>(a.partials, (split * a.outs + row) * a.cols + col, n, acc[o][i]);
            else finish4(a, row * a.cols + col, n, acc[o][i]);
        }
    }
}

// The splits' sums added in order: four elements per thread.
__global__ __launch_bounds__(256) void weight_join_kernel(WeightGrad a) {
    const int64_t size = a.outs * a.cols;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= size) return;
    const int n = (int)min((int64_t)4, size - at);
    v4f sum = read4<ZERO_F32>(a.partials, at, n);
#pragma unroll 4
    for (int s = 1; s < a.splits; ++s) {
        const v4f x = read4<ZERO_F32>(a.partials, s * size + at, n);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[k] += x[k];
    }
    finish4(a, at, n, sum);
}

template <int DT>
int launch_dt(const WeightGrad& a, hipStream_t s) {
    const dim3 grid((uint32_t)(a.tiles * a.splits));
    if (a.tile == 256) weight_grad_kernel<DT, 256, 256, 2, 4><<<grid, 512, 0, s>>>(a);
    else weight_grad_kernel<DT, 128, 128, 2, 2><<<grid, 256, 0, s>>>(a);
    return (int)hipGetLastError();
}

}  // namespace

int launch_weight_grad(const WeightGrad& l, int dtype, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (const int e = dtype == ZERO_BF16 ? launch_dt<ZERO_BF16>(l, s) : launch_dt<ZERO_F16>(l, s)) return e;
    if (l.partials) {
        const int64_t quads = (l.outs * l.cols + 3) / 4;
        weight_join_kernel<<<(uint32_t)((quads + 255) / 256), 256, 0, s>>>(l);
        return (int)hipGetLastError();
    }
    return 0;
}

}  // namespace zf
