// zeroflat_act.hip -- gfx950 (MI355X, CDNA4, wave64) kernels of activations kept
// in 8 bits:
//   act_forward_kernel   the 8-bit checkpoint of a matrix; with an activation
//                        function also its output, and the gate's factor
//   act_backward_kernel  a checkpoint restored, or the activation's gradient
//                        taken from it, with the output's checkpoint made anew
//
// A checkpoint is int8 codes, rows padded with zeros to blocks of 32, and one
// exponent E per block, a value being code * 2^(E - 133): E from the block's
// largest magnitude, so that it lies in [64, 128) units of a code (the OCP
// Microscaling formats' rule for shared exponents).  The scale is a power of
// two because code * 2^k is exact in bf16 and in fp16's range: the
// matrix cores multiply restored values without another rounding.  It costs up
// to one bit of a code against a scale of largest/127.
//
// A lane holds eight columns, four lanes a block: its maximum takes two lane
// exchanges.  All of it is bound by memory, every array once; 16-byte loads and
// stores at any element offset, 8-byte ones for codes, which go past the caches: they
// are read again a whole backward pass later.  bf16, at the rate of what they must
// move: the checkpoint of 16384 x 4096 in 37.5 us (5.4 TB/s), the gated forward pass
// over 8192 x 11008 in 118 us (6.1 TB/s; 122 with the codes cached), its backward pass in
// 118 us (6.2 TB/s; 125 with the gradients cached).
#include "zf_vec.h"

namespace zf {
namespace {

constexpr int kThreads = 256;
constexpr int kNan = 255;                      // the exponent of a block with an infinity or a NaN
constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float pow2(uint32_t biased) { return __uint_as_float(biased << 23); }
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float fma32(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
// clamped, a NaN kept
__device__ __forceinline__ float within(float x, float most) {
    return x > most ? most : x < -most ? -most : x;
}

// ---------------------------------------------------------------- functions
// 1 / (1 + e^-x): the exponential overflows to infinity and the quotient to 0.
__device__ __forceinline__ float logistic(float x) { return rcp_hw(1.0f + exp2_hw(-kLog2e * x)); }

// The normal distribution's P(X < x) and density at x.  For z = |x| / sqrt 2,
// erfc(z) = e^(-z^2) t P(t) with t = 1 / (1 + z/2), P fitted by weighted least
// squares to e^(z^2) erfc(z) on 0 <= z <= 10.3 (relative error 5e-8); the tail
// keeps its relative accuracy, and the exponential is the density's too.
__device__ __forceinline__ void normal(float x, float& cdf, float& density) {
    const float t = rcp_hw(fma32(fabsf(x), 0.35355339059327376f, 1.0f));
    float p = -0.05914958566427231f;
    p = fma32(p, t, 0.2849690914154053f);
    p = fma32(p, t, -0.4880177080631256f);
    p = fma32(p, t, 0.27900487184524536f);
    p = fma32(p, t, -0.027273206040263176f);
    p = fma32(p, t, 0.20296156406402588f);
    p = fma32(p, t, 0.24303415417671204f);
    p = fma32(p, t, 0.2823849022388458f);
    p = fma32(p, t, 0.2820858657360077f);
    const float e = exp2_hw((-0.5f * kLog2e) * x * x);
    const float tail = 0.5f * e * (p * t);
    cdf = x < 0.0f ? tail : 1.0f - tail;
    density = e * 0.3989422804014327f;
}

// act(x) and act'(x).  Beyond the clamps the functions are 0 or x to every bit
// of fp32, and squares and cubes inside cannot overflow to 0 * inf; a NaN comes
// through both.
template <int KIND>
__device__ __forceinline__ void act(float x, float& y, float& slope) {
    if constexpr (KIND == ZERO_SILU) {
        const float s = logistic(x);
        y = x * s;
        slope = s * fma32(within(x, 200.0f), 1.0f - s, 1.0f);
    } else if constexpr (KIND == ZERO_GELU) {
        const float c = within(x, 40.0f);
        float cdf, density;
        normal(c, cdf, density);
        y = x * cdf;
        slope = fma32(c, density, cdf);
    } else {
        constexpr float c2 = 1.5957691216057308f, a = 0.044715f;   // 2 sqrt(2 / pi)
        const float c = within(x, 20.0f), sq = c * c;
        const float s = logistic(c2 * c * fma32(a, sq, 1.0f));     // 0.5 (1 + tanh u) = logistic(2 u)
        y = x * s;
        slope = fma32(c * s * (1.0f - s), c2 * fma32(3.0f * a, sq, 1.0f), s);
    }
}

// ---------------------------------------------------------------- checkpoints
// The maximum over a block's four lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0xB1, 0xf, 0xf, false));   // lanes 1 0 3 2
    return max(x, (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, 0x4E, 0xf, 0xf, false)); // lanes 2 3 0 1
}

// The codes of eight columns (0 beyond the matrix) and their block's exponent.
// All four lanes of a block take part.
__device__ __forceinline__ void quantise(const float (&x)[8], int least, v2u& codes, uint32_t& exponent) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
    top = quad_max(top);
    const bool bad = top >= 0x7f800000u;
    const uint32_t e = max(top >> 23, (uint32_t)least);
    exponent = bad ? (uint32_t)kNan : e;
    const float inv = pow2(260u - e);              // 2^(133 - E), E of 7 .. 254
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // a product with a power of two is exact; ties to even
            const float q = fminf(fmaxf(__builtin_rintf(x[4 * h + k] * inv), -127.0f), 127.0f);
            w |= (uint32_t)((int)q & 0xff) << (8 * k);
        }
        codes[h] = bad ? 0u : w;
    }
}
__device__ __forceinline__ void restore(v2u codes, uint32_t exponent, float (&x)[8]) {
    const float s = exponent == (uint32_t)kNan ? __uint_as_float(0x7fc00000u) : pow2(exponent - 6u);
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = (float)(int8_t)(codes[k / 4] >> (8 * (k % 4))) * s;
}

struct Place {
    uint32_t row, group;     // of the launch's rows; eight columns each
    int col, n;              // n <= 0: padding only
};
__device__ __forceinline__ Place place_of(uint32_t g, const Div& per_row, int64_t cols) {
    Place p;
    p.row = div_by(g, per_row);
    p.group = g - p.row * per_row.d;
    p.col = (int)(p.group * 8);
    p.n = (int)min((int64_t)8, cols - p.col);
    return p;
}
__device__ __forceinline__ void keep(const float (&x)[8], int least, int8_t* codes, uint8_t* exponents,
                                     uint32_t g, int stream) {
    v2u c;
    uint32_t e;
    quantise(x, least, c, e);
    if (stream) {
        ZF_APART;
        __builtin_nontemporal_store(c, reinterpret_cast<v2u*>(codes) + g);
        ZF_APART;
    } else {
        reinterpret_cast<v2u*>(codes)[g] = c;
    }
    if ((g & 3) == 0) exponents[g >> 2] = (uint8_t)e;
}

// ---------------------------------------------------------------- kernels
template <int DT, int KIND, bool GATED>
__global__ __launch_bounds__(kThreads) void act_forward_kernel(ActLaunch a) {
    // a block's four lanes are in or out together: groups in a row are a multiple of four
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= a.groups) return;
    const Place p = place_of(g, a.per_row, a.cols);
    float x[8];
    load8<DT>(a.x, (int64_t)p.row * a.x_ld + p.col, p.n, x);
    float u[8];
    if constexpr (GATED) load8<DT>(a.up, (int64_t)p.row * a.up_ld + p.col, p.n, u);
    keep(x, a.least, a.codes, a.exponents, g, 1);
    if constexpr (GATED) keep(u, a.least, a.up_codes, a.up_exponents, g, 1);
    if constexpr (KIND >= 0) {
        if (p.n <= 0) return;
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float slope;
            act<KIND>(x[k], y[k], slope);
            if constexpr (GATED) y[k] *= u[k];
        }
        store8<DT>(a.y, (int64_t)p.row * a.y_ld + p.col, p.n, y, a.stream);
    }
}

template <int DT, int KIND, bool GATED>
__global__ __launch_bounds__(kThreads) void act_backward_kernel(ActLaunch a) {
    const uint32_t g = blockIdx.x * kThreads + threadIdx.x;
    if (g >= a.groups) return;
    const Place p = place_of(g, a.per_row, a.cols);
    float x[8], u[8], d[8];
    if constexpr (KIND >= 0) load8<DT>(a.x, (int64_t)p.row * a.x_ld + p.col, p.n, d);
    const v2u cx = reinterpret_cast<const v2u*>(a.codes)[g];
    const uint32_t ex = a.exponents[g >> 2];
    restore(cx, ex, x);
    if constexpr (GATED) {
        const v2u cu = reinterpret_cast<const v2u*>(a.up_codes)[g];
        restore(cu, a.up_exponents[g >> 2], u);
    }
    if constexpr (KIND < 0) {
        if (p.n > 0) store8<DT>(a.y, (int64_t)p.row * a.y_ld + p.col, p.n, x, a.stream);
    } else {
        float dx[8], du[8], y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float slope;
            act<KIND>(x[k], y[k], slope);
            if constexpr (GATED) {
                dx[k] = d[k] * u[k] * slope;
                du[k] = d[k] * y[k];
                y[k] *= u[k];
            } else {
                dx[k] = d[k] * slope;
            }
        }
        if (p.n > 0) {
            store8<DT>(a.y, (int64_t)p.row * a.y_ld + p.col, p.n, dx, a.stream);
            if constexpr (GATED) store8<DT>(a.dup, (int64_t)p.row * a.dup_ld + p.col, p.n, du, a.stream);
        }
        if (a.again_codes) {
            // columns beyond the matrix stand for 0 whatever the function makes of 0; the
            // codes stay cached for the weight gradient that reads them next.  Cached and
            // past the caches, us, bf16, alone: gated 8192 x 11008 135, 132 (118 without
            // them), 16384 x 4096 98, 95, plain 66, 59; with that weight gradient (1024
            // outputs) 345, 349; 236, 239; 204, 206; gated 4096 x 4096 80, 85.
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = k < p.n ? y[k] : 0.0f;
            keep(y, a.least, a.again_codes, a.again_exponents, g, 0);
        }
    }
}

template <int DT, int KIND>
void act_of(const ActLaunch& a, bool backward, dim3 grid, hipStream_t s) {
    if constexpr (KIND >= 0) {
        if (a.up_codes) {
            if (backward) act_backward_kernel<DT, KIND, true><<<grid, kThreads, 0, s>>>(a);
            else act_forward_kernel<DT, KIND, true><<<grid, kThreads, 0, s>>>(a);
            return;
        }
    }
    if (backward) act_backward_kernel<DT, KIND, false><<<grid, kThreads, 0, s>>>(a);
    else act_forward_kernel<DT, KIND, false><<<grid, kThreads, 0, s>>>(a);
}
template <int DT>
void act_dt(const ActLaunch& a, bool backward, dim3 grid, hipStream_t s) {
    if (a.kind < 0) act_of<DT, -1>(a, backward, grid, s);
    else if (a.kind == ZERO_GELU) act_of<DT, ZERO_GELU>(a, backward, grid, s);
    else if (a.kind == ZERO_GELU_TANH) act_of<DT, ZERO_GELU_TANH>(a, backward, grid, s);
    else act_of<DT, ZERO_SILU>(a, backward, grid, s);
}

template <typename T>
T* moved(T* p, int64_t bytes) {
    return p ? reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + bytes) : nullptr;
}

}  // namespace

int launch_act(const ActLaunch& l, int backward, void* stream) {
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t per_row = (l.cols + 31) / 32 * 4, size = l.dtype == ZERO_F32 ? 4 : 2;
    // groups are counted in 31 bits: larger matrices take several launches
    const int64_t most = ((int64_t)1 << 30) / per_row;
    // Large outputs go past the caches, but for fp32 where a call writes more than it
    // reads: cached and past the caches, us, 65536 x 1024, restore 61, 95, gated backward
    // 169, 217, x 1023 76, 97 and 194, 206; forward 104, 94, gated 118, 108, backward 105, 105.
    const bool cached = l.dtype == ZERO_F32 && backward && (l.kind < 0 || l.dup);
    for (int64_t r = 0; r < l.rows; r += most) {
        const int64_t n = l.rows - r < most ? l.rows - r : most;
        ActLaunch a = l;
        a.per_row = make_div((uint32_t)per_row);
        a.stream = !cached && streams(l.rows * l.cols * size * (l.dup ? 2 : 1));
        a.groups = (uint32_t)(n * per_row);
        a.x = moved(l.x, r * l.x_ld * size);
        a.up = moved(l.up, r * l.up_ld * size);
        a.y = moved(l.y, r * l.y_ld * size);
        a.dup = moved(l.dup, r * l.dup_ld * size);
        a.codes = moved(l.codes, r * per_row * 8);
        a.up_codes = moved(l.up_codes, r * per_row * 8);
        a.again_codes = moved(l.again_codes, r * per_row * 8);
        a.exponents = moved(l.exponents, r * per_row / 4);
        a.up_exponents = moved(l.up_exponents, r * per_row / 4);
        a.again_exponents = moved(l.again_exponents, r * per_row / 4);
        const dim3 grid((a.groups + kThreads - 1) / kThreads);
        if (a.dtype == ZERO_F32) act_dt<ZERO_F32>(a, backward, grid, s);
        else if (a.dtype == ZERO_F16) act_dt<ZERO_F16>(a, backward, grid, s);
        else act_dt<ZERO_BF16>(a, backward, grid, s);
        if (const int e = (int)hipGetLastError()) return e;
    }
    return 0;
}

}  // namespace zf
