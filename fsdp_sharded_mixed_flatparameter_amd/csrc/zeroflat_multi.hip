// zeroflat_multi.hip -- gfx950 (MI355X, CDNA4, wave64) kernels of the step
// over a list of tensors:
//   multi_stats_kernel  sums of squares of the unscaled gradients, per span of
//                       a tensor
//   multi_fold_kernel   those sums per tensor and over all; for a step also its
//                       scalars, loss scaler and counters (multi_prepare_kernel
//                       does only that)
//   multi_adamw_kernel  AdamW with 32-bit or 8-bit states, 16-bit copy
//   multi_adamw_short_kernel  the same for short lists, with the fold inside
//
// A step reads the gradients twice and everything else once; none of it is a
// contraction.  The state
// arenas are rows of 256 elements, so a wave owns whole rows: in a row lane l
// holds elements 4l .. 4l+3 (16 bytes of each fp32 array, 8 of a 16-bit one,
// 4 of an 8-bit one per lane).  Only the gradients and the 16-bit parameters
// lie elsewhere, at any element offset; the plan's tables say which tensor a
// tile (of rows) or a span (of gradient elements) belongs to.
//
// Built with -ffp-contract=off and correctly rounded fp32 division and square
// root, as the flat step's kernels; the 32-bit form repeats their operation
// order, so a list of one tensor gives the flat step's bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "zf_launch.h"

namespace zf {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRow = ZERO_ROW;
static_assert(kRow == 256, "one quad per lane and row");

typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
// fp32 gradients may start at any element: quads of 4-byte alignment
typedef float v4f_a4 __attribute__((ext_vector_type(4), aligned(4)));

// The plan's tables do not change while a kernel runs: reading them through
// the constant address space keeps wave-uniform reads scalar.
#define ZF_CONST __attribute__((address_space(4)))
template <typename T>
__device__ __forceinline__ const ZF_CONST T* as_const(const T* p) {
    return (const ZF_CONST T*)(uintptr_t)p;
}

template <typename T>
__device__ __forceinline__ T ldnt(const void* p) {
    return __builtin_nontemporal_load(static_cast<const T*>(p));
}
template <typename T>
__device__ __forceinline__ void stnt(void* p, T x) {
    __builtin_nontemporal_store(x, static_cast<T*>(p));
}

// ---------------------------------------------------------------- formats
__device__ __forceinline__ float h2f(uint32_t h) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h);
}
__device__ __forceinline__ float b2f(uint32_t h) { return __uint_as_float(h << 16); }
template <int DT>
__device__ __forceinline__ float cvt16(uint32_t h) {
    return DT == ZERO_F16 ? h2f(h) : b2f(h);
}
// To binary16 / bfloat16, to nearest, ties to even.  binary16 by the scalar
// conversion, one instruction per value (the packed one does not always round
// to nearest); bfloat16 on the bit patterns.  Rounding on the bit patterns
// alone, as the flat step does it, is 14 instructions per value for binary16,
// which the 8-bit form has no time for.
template <int DT>
__device__ __forceinline__ uint32_t round16(float x) {
    if constexpr (DT == ZERO_F16) {
        uint32_t h;
        asm("v_cvt_f16_f32 %0, %1" : "=v"(h) : "v"(x));
        return x != x ? ((h & 0x8000u) | 0x7e00u) : h;   // the quiet NaN
    } else {
        const uint32_t u = __float_as_uint(x);
        if (x != x) return ((u >> 16) & 0x8000u) | 0x7fc0u;
        return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
    }
}
template <int DT>
__device__ __forceinline__ float load_one(const void* p, int64_t i) {
    if constexpr (DT == ZERO_F32) return static_cast<const float*>(p)[i];
    else return cvt16<DT>(static_cast<const uint16_t*>(p)[i]);
}

// ---------------------------------------------------------------- lanes
// DPP wave shifts (gfx9-family controls): the neighbour's value, `edge` in the
// lane that has none.
constexpr int kDppWaveShl1 = 0x130, kDppWaveShr1 = 0x138;
__device__ __forceinline__ uint32_t from_above(uint32_t x, uint32_t edge) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)edge, (int)x, kDppWaveShl1, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t from_below(uint32_t x, uint32_t edge) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)edge, (int)x, kDppWaveShr1, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}
// Reductions over a wave: DPP shifts within rows of 16 lanes, then the row
// broadcasts (gfx9-family controls, 0 where there is no source); lane 63 ends
// with all of it.  A butterfly through LDS permutes takes three times as long,
// 0.3 us of a small kernel.
#define ZF_WAVE_STEPS(STEP)                                                          \
    STEP(0x111, 0xf) /* row_shr:1 */ STEP(0x112, 0xf) /* row_shr:2 */                \
    STEP(0x114, 0xf) /* row_shr:4 */ STEP(0x118, 0xf) /* row_shr:8 */                \
    STEP(0x142, 0xa) /* row_bcast:15 */ STEP(0x143, 0xc) /* row_bcast:31 */
#define ZF_DPP(x, ctrl, rows) __builtin_amdgcn_update_dpp(0, (int)(x), ctrl, rows, 0xf, false)
// The sum in a fixed order, in every lane.
__device__ __forceinline__ double wave_sum(double x) {
#define ZF_SUM_STEP(ctrl, rows)                                                      \
    {                                                                                \
        const uint64_t b = __builtin_bit_cast(uint64_t, x);                          \
        const uint64_t o = (uint64_t)(uint32_t)ZF_DPP((uint32_t)b, ctrl, rows) |     \
                           (uint64_t)(uint32_t)ZF_DPP(b >> 32, ctrl, rows) << 32;    \
        x += __builtin_bit_cast(double, o);                                          \
    }
    ZF_WAVE_STEPS(ZF_SUM_STEP)
#undef ZF_SUM_STEP
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)lane_value((uint32_t)b, 63) |
                                          (uint64_t)lane_value((uint32_t)(b >> 32), 63) << 32);
}
// The largest of values that are neither negative nor NaN (whose patterns are
// ordered as integers), as a scalar.
__device__ __forceinline__ float wave_max(float x) {
    uint32_t u = __float_as_uint(x);
#define ZF_MAX_STEP(ctrl, rows)                            \
    {                                                      \
        const uint32_t o = (uint32_t)ZF_DPP(u, ctrl, rows); \
        u = u > o ? u : o;                                 \
    }
    ZF_WAVE_STEPS(ZF_MAX_STEP)
#undef ZF_MAX_STEP
    return __uint_as_float(lane_value(u, 63));
}
// fixed order; valid in thread 0
template <int WAVES>
__device__ __forceinline__ double block_sum(double x) {
    __shared__ double sh[WAVES];
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = x;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < WAVES; ++w) t += sh[w];
    }
    return t;
}

// ---------------------------------------------------------------- step scalars
// A bijection of 32-bit numbers whose output bits depend on every input bit; the
// shifts and multipliers are C. Wellons' ("Prospecting for Hash Functions",
// 2018, found by a search for the least bias).
__device__ __forceinline__ uint32_t mix(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x7FEB352Du;
    h = (h ^ (h >> 15)) * 0x846CA68Bu;
    return h ^ (h >> 16);
}
// The scalars of the step state.
__device__ __forceinline__ MultiState read_state(const zero_step_state_t* st) {
    return {st->sumsq, st->remote_sumsq, st->beta1_pow, st->beta2_pow, st->loss_scale, st->min_scale,
            st->overflow, st->remote_overflow, st->dynamic, st->window, st->good_steps, st->step};
}
__device__ __forceinline__ void add_sum(MultiState& st, double sum, int reset) {
    const int bad = !isfinite(sum);
    st.sumsq = reset ? sum : st.sumsq + sum;
    st.overflow = reset ? bad : st.overflow | bad;
}
// What the update needs of them: skip, clip, unscale and bias corrections with
// t = step + 1 as the flat step has them, the 8-bit form's factors and the key
// of its random numbers.
__device__ __forceinline__ MultiScalars step_scalars(const MultiStep& p, const MultiState& st) {
    MultiScalars r;
    r.skip = (st.overflow | st.remote_overflow) != 0;
    r.norm = sqrt(st.sumsq + st.remote_sumsq);
    r.coef = 1.0f;
    if (p.max_norm > 0.0) {
        const double c = p.max_norm / (r.norm + 1e-6);
        r.coef = (float)(c < 1.0 ? c : 1.0);
    }
    r.inv = (float)(1.0 / (double)st.loss_scale);
    const double bc1 = 1.0 - st.beta1_pow * p.beta1, bc2 = 1.0 - st.beta2_pow * p.beta2;
    r.bc1 = (float)bc1;
    r.bc2 = (float)bc2;
    r.rs = (float)(1.0 / sqrt(bc2));
    r.lr = p.lr;
    r.lr_bc1 = p.lr / bc1;
    r.wd = p.wd;
    r.key = mix((uint32_t)st.step + 1u + p.seed);
    return r;
}
// The state after the step: the loss scaler and the counters as the flat step
// moves them; without p.advance only the statistics of `old`.  One thread.
__device__ __forceinline__ void write_state(const MultiStep& p, const MultiState& old,
                                            const MultiScalars& r) {
    zero_step_state_t* st = p.st;
    if (!p.advance) {
        st->sumsq = old.sumsq;
        st->overflow = old.overflow;
        return;
    }
    st->last_norm = r.norm;
    st->last_skipped = r.skip;
    st->last_coef = r.skip ? 0.0f : r.coef;
    if (r.skip) {
        if (old.dynamic) {
            const float h = old.loss_scale / 2.0f;
            st->loss_scale = h > old.min_scale ? h : old.min_scale;
        }
        st->good_steps = 0;
    } else {
        st->step = old.step + 1;
        st->beta1_pow = old.beta1_pow * p.beta1;
        st->beta2_pow = old.beta2_pow * p.beta2;
        if (old.dynamic) {
            const bool grow = old.good_steps + 1 == old.window;
            if (grow && old.loss_scale < 0x1p127f) st->loss_scale = old.loss_scale * 2.0f;
            st->good_steps = grow ? 0 : old.good_steps + 1;
        }
    }
    st->sumsq = 0.0;
    st->overflow = 0;
}

// ---------------------------------------------------------------- statistics
// One block per span: E consecutive elements of one tensor, from the tensor's
// first 16-byte boundary on (the first span also takes the elements before it,
// the last one what is left).  Squares and sums in fp64, where the square of
// an fp32 value is exact.
constexpr int kStatU = 8;   // 16-byte loads in flight per thread
// The pass streams with non-temporal loads, except that before an update it
// leaves the first gradients, up to the size of the memory-side cache, where
// the update finds them again: the 2.02e8-element bf16 block's step took 957 us
// with none kept, 944 with 128 MiB, 930 with 256 and 933 with all of it (405
// MB), the 1.25e9-element fp16 shard's 3613, 3599, 3594 and 3754.  On its own
// the pass is 16% slower with plain loads (72 against 62 us).
constexpr int64_t kKeepBytes = (int64_t)256 << 20;

template <int DT>
__device__ __forceinline__ void add_squares(v4u w, double& s0, double& s1) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == ZERO_F32) {
            const double d = (double)__uint_as_float(x[i]);
            if (i & 1) s1 = __builtin_fma(d, d, s1);
            else s0 = __builtin_fma(d, d, s0);
        } else {
            const double a = (double)cvt16<DT>(x[i] & 0xffffu);
            const double b = (double)cvt16<DT>(x[i] >> 16);
            s0 = __builtin_fma(a, a, s0);
            s1 = __builtin_fma(b, b, s1);
        }
    }
}

template <int DT, bool KEEP>
__device__ __forceinline__ void sum_vectors(const char* base, int nvec, double& s0, double& s1) {
    const int tid = threadIdx.x;
    auto load = [&](int i) {
        const char* p = base + 16 * (int64_t)i;
        return KEEP ? *reinterpret_cast<const v4u*>(p) : ldnt<v4u>(p);
    };
    int v = 0;
    for (; v + kThreads * kStatU <= nvec; v += kThreads * kStatU) {
        v4u w[kStatU];
#pragma unroll
        for (int u = 0; u < kStatU; ++u) w[u] = load(v + u * kThreads + tid);
#pragma unroll
        for (int u = 0; u < kStatU; ++u) add_squares<DT>(w[u], s0, s1);
    }
    if (v < nvec) {
        v4u w[kStatU];
#pragma unroll
        for (int u = 0; u < kStatU; ++u) {
            const int i = v + u * kThreads + tid;
            w[u] = i < nvec ? load(i) : v4u{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int u = 0; u < kStatU; ++u) add_squares<DT>(w[u], s0, s1);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) multi_stats_kernel(MultiNormLaunch a) {
    constexpr int kEs = DT == ZERO_F32 ? 4 : 2;
    constexpr int kV = 16 / kEs;   // elements per 16-byte load
    const int s = blockIdx.x;
    if (s == 0 && threadIdx.x == 0 && a.snapshot) *a.snapshot = read_state(a.st);
    const double inv = 1.0 / (double)as_const(a.st)->loss_scale;
    const int k = as_const(a.span_tensor)[s];
    const ZF_CONST MultiEntry* e = as_const(a.entries) + k;
    const char* g = static_cast<const char*>(e->grad);
    const int64_t n = e->numel;
    const int local = s - e->span0;
    const bool last = local == e->n_spans - 1;
    int64_t head = (int64_t)((16 - ((uintptr_t)g & 15)) & 15) / kEs;
    if (head > n) head = n;
    int64_t lo = head + (int64_t)local * a.span;
    if (lo > n) lo = n;
    int64_t hi = lo + a.span;
    if (hi > n || last) hi = n;
    const char* base = g + lo * kEs;
    const int nvec = (int)((hi - lo) / kV);   // a span holds at most 2^31 elements
    const int tid = threadIdx.x;
    double s0 = 0.0, s1 = 0.0;
    if (s < a.keep_spans) sum_vectors<DT, true>(base, nvec, s0, s1);
    else sum_vectors<DT, false>(base, nvec, s0, s1);
    // fewer than kV elements after the last vector, fewer than kV before the first
    const int64_t rest = lo + (int64_t)nvec * kV + tid;
    if (rest < hi) {
        const double d = (double)load_one<DT>(g, rest);
        s0 = __builtin_fma(d, d, s0);
    }
    if (local == 0 && tid < head) {
        const double d = (double)load_one<DT>(g, tid);
        s1 = __builtin_fma(d, d, s1);
    }
    const double sum = block_sum<kWaves>(s0 + s1);
    // the loss scale, a power of two, is applied to the sum as exactly as to
    // every element
    if (tid == 0) a.partials[s] = sum * inv * inv;
}

// ---------------------------------------------------------------- folds
// Block 0: the total, and with `step` what the update needs of it; the other
// blocks: a tensor's sum each, or (per_wave) a tensor's sum per wave.  A launch
// of its own: folding in the block that finishes last instead (stores and a
// count at device scope) made the small MLP's statistics 8.3 us against 6.0 and
// the 2.02e8-element block's 70 against 66, and a count per block of the update
// costs about 12 ns each, one after the other.
constexpr int kFoldThreads = 512;
__device__ __forceinline__ void fold(const MultiNormLaunch& a, const MultiStep* step, int per_wave) {
    int p0 = 0, np = a.n_spans;
    // read first: thread 0's chain is the whole launch
    MultiState st = {};
    if (blockIdx.x == 0 && threadIdx.x == 0) st = read_state(a.st);
    if (per_wave && blockIdx.x > 0) {
        const int k = (int)(blockIdx.x - 1) * (kFoldThreads / 64) +
                      __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
        if (k >= a.n_tensors) return;
        p0 = as_const(a.entries)[k].span0;
        np = as_const(a.entries)[k].n_spans;
        double x = 0.0;
        for (int i = threadIdx.x & 63; i < np; i += 64) x += a.partials[p0 + i];
        x = wave_sum(x);
        if ((threadIdx.x & 63) == 0) a.tensor_sumsq[k] = x;
        return;
    }
    if (blockIdx.x > 0) {
        p0 = a.entries[blockIdx.x - 1].span0;
        np = a.entries[blockIdx.x - 1].n_spans;
    }
    double x = 0.0;
    for (int i = threadIdx.x; i < np; i += kFoldThreads * kStatU) {
        double v[kStatU];
#pragma unroll
        for (int u = 0; u < kStatU; ++u) {
            const int j = i + u * kFoldThreads;
            v[u] = j < np ? a.partials[p0 + j] : 0.0;
        }
#pragma unroll
        for (int u = 0; u < kStatU; ++u) x += v[u];
    }
    x = block_sum<kFoldThreads / 64>(x);
    if (threadIdx.x != 0) return;
    if (blockIdx.x > 0) {
        a.tensor_sumsq[blockIdx.x - 1] = x;
        return;
    }
    add_sum(st, x, a.reset);
    if (step) {
        const MultiScalars r = step_scalars(*step, st);
        *step->scalars = r;
        write_state(*step, st, r);
    } else {
        a.st->sumsq = st.sumsq;
        a.st->overflow = st.overflow;
    }
}
__global__ void __launch_bounds__(kFoldThreads) multi_fold_kernel(MultiNormLaunch a, int per_wave) {
    fold(a, nullptr, per_wave);
}
__global__ void __launch_bounds__(kFoldThreads) multi_fold_step_kernel(MultiNormLaunch a,
                                                                       MultiStep step, int per_wave) {
    fold(a, &step, per_wave);
}
__global__ void multi_prepare_kernel(MultiStep step) {
    if (threadIdx.x != 0) return;
    const MultiState st = read_state(step.st);
    const MultiScalars r = step_scalars(step, st);
    *step.scalars = r;
    write_state(step, st, r);
}

// the record of an earlier launch, by scalar loads
template <typename T>
__device__ __forceinline__ T load_record(const T* p) {
    static_assert(sizeof(T) % 8 == 0, "read in 8-byte pieces");
    uint64_t w[sizeof(T) / 8];
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 8); ++i)
        w[i] = as_const(reinterpret_cast<const uint64_t*>(p))[i];
    T t;
    __builtin_memcpy(&t, w, sizeof t);
    return t;
}
struct TensorScalars {
    float rate, keep;
};
template <int BITS>
__device__ __forceinline__ TensorScalars tensor_scalars(const MultiScalars& s,
                                                        const ZF_CONST MultiEntry* e) {
    TensorScalars t;
    t.keep = (float)(1.0 - s.lr * e->lr_mult * (s.wd * e->decay_mult));
    t.rate = (float)((BITS == 8 ? s.lr_bc1 : s.lr) * e->lr_mult);
    return t;
}

// ---------------------------------------------------------------- 8-bit codes
constexpr float kMost4 = 448.0f, kMost5 = 57344.0f;
__device__ __forceinline__ float row_scale(float top, float most_inv) {
    return top > 0.0f ? fmaxf(fminf(top, 0x1.fffffep127f) * most_inv, 0x1p-126f) : 0.0f;
}
// 1/x to the nearest, for a scale (2^-126 to 2^120, so x and 1/x are normal):
// one step of Newton's method from the 1-ulp instruction, checked for every
// mantissa against the IEEE quotient; a quarter of the division's instructions.
__device__ __forceinline__ float reciprocal(float x) {
    const float r = __builtin_amdgcn_rcpf(x);
    return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}
// Four second moments (times 1/scale) as e5m2, rounded with the row's numbers.
// e5m2's exponent is fp32's less 112; the difference, modulo the 6 exponent
// bits that are kept, is added before the cut.  The largest, 57344, has no bit
// below the cut, so nothing added carries past it.
__device__ __forceinline__ uint32_t round_e5m2(const float v[4], float inv, uint32_t key, int lane) {
    const uint32_t h = mix(key + (uint32_t)lane * 0x9E3779B9u);
    uint32_t k = h * 0x2C1B3C6Du;
    k ^= k >> 13;
    constexpr uint32_t kMask = 0xffffu << 5, kBias = (uint32_t)(64 - 48) << 23;
    const uint32_t r[4] = {(h << 5) & kMask, (h >> 11) & kMask, (k << 5) & kMask, (k >> 11) & kMask};
    uint32_t out = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float y = __builtin_amdgcn_fmed3f(v[c] * inv, 0x1p-14f, kMost5);
        const uint32_t q = ((__float_as_uint(y) + r[c] + kBias) >> 21) & 0xffu;
        out |= (v[c] > 0.0f ? q : 0u) << (8 * c);
    }
    return out;
}

// ---------------------------------------------------------------- the update
// One lane's quad of one row.  m, v hold fp32 values or, with 8-bit states,
// four codes in their first word.
template <int BITS>
struct Quad {
    float p[4];
    v4u m, v;          // BITS 8: .x only
};
template <int BITS>
__device__ __forceinline__ void load_state(const MultiAdamLaunch& a, int64_t i, Quad<BITS>& q) {
    const v4f x = ldnt<v4f>(a.p + i);
    q.p[0] = x.x; q.p[1] = x.y; q.p[2] = x.z; q.p[3] = x.w;
    if constexpr (BITS == 32) {
        q.m = ldnt<v4u>(static_cast<const float*>(a.m) + i);
        q.v = ldnt<v4u>(static_cast<const float*>(a.v) + i);
    } else {
        q.m.x = ldnt<uint32_t>(static_cast<const uint8_t*>(a.m) + i);
        q.v.x = ldnt<uint32_t>(static_cast<const uint8_t*>(a.v) + i);
    }
}
template <int BITS>
__device__ __forceinline__ void store_state(const MultiAdamLaunch& a, int64_t i, const Quad<BITS>& q) {
    stnt<v4f>(a.p + i, v4f{q.p[0], q.p[1], q.p[2], q.p[3]});
    if constexpr (BITS == 32) {
        stnt<v4u>(static_cast<float*>(a.m) + i, q.m);
        stnt<v4u>(static_cast<float*>(a.v) + i, q.v);
    } else {
        stnt<uint32_t>(static_cast<uint8_t*>(a.m) + i, q.m.x);
        stnt<uint32_t>(static_cast<uint8_t*>(a.v) + i, q.v.x);
    }
}

// The update of a row's quads, in place; ms / vs: the row's scales (8-bit).
template <int BITS>
__device__ __forceinline__ void update_quad(const MultiAdamLaunch& a, const MultiScalars& s,
                                            const TensorScalars& t, const float gv[4],
                                            Quad<BITS>& q, float& ms, float& vs, uint32_t key,
                                            int lane) {
    if constexpr (BITS == 32) {
        float m[4] = {__uint_as_float(q.m.x), __uint_as_float(q.m.y), __uint_as_float(q.m.z),
                      __uint_as_float(q.m.w)};
        float v[4] = {__uint_as_float(q.v.x), __uint_as_float(q.v.y), __uint_as_float(q.v.z),
                      __uint_as_float(q.v.w)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float u = gv[c] * s.inv;
            const float g = u * s.coef;
            m[c] = a.b1 * m[c] + a.c1 * g;
            v[c] = a.b2 * v[c] + a.c2 * (g * g);
            const float mh = m[c] / s.bc1;
            const float vh = v[c] / s.bc2;
            const float d = sqrtf(vh) + a.eps;
            q.p[c] = q.p[c] * t.keep - (t.rate * mh) / d;
        }
        q.m = v4u{__float_as_uint(m[0]), __float_as_uint(m[1]), __float_as_uint(m[2]),
                  __float_as_uint(m[3])};
        q.v = v4u{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                  __float_as_uint(v[3])};
    } else {
        typedef float v2f __attribute__((ext_vector_type(2)));
        const v2f m01 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.m.x, false);
        const v2f m23 = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.m.x, true);
        const v2f v01 = __builtin_amdgcn_cvt_pk_f32_bf8((int)q.v.x, false);
        const v2f v23 = __builtin_amdgcn_cvt_pk_f32_bf8((int)q.v.x, true);
        float m[4] = {m01.x, m01.y, m23.x, m23.y}, v[4] = {v01.x, v01.y, v23.x, v23.y};
        float tm = 0.0f, tv = 0.0f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            // the states' operations are rounded one by one, so that they are
            // the same on any machine: a random rounding that falls the other
            // way is a whole code off.  Two products for g: the factors' own may
            // be below fp32's normal numbers (a scale near 2^127 with a clip
            // below one) and lose the gradient
            const float u = gv[c] * s.inv;
            const float g = u * s.coef;
            m[c] = a.b1 * (m[c] * ms) + a.c1 * g;
            v[c] = a.b2 * (v[c] * vs) + a.c2 * (g * g);
            // the parameter's are not held in 8 bits: fused, and by the root
            // and the reciprocal instructions (1 unit in the last place each
            // of a step that is far smaller than the parameter)
            const float d = __builtin_fmaf(__builtin_amdgcn_sqrtf(v[c]), s.rs, a.eps);
            q.p[c] = __builtin_fmaf(q.p[c], t.keep, -((t.rate * m[c]) * __builtin_amdgcn_rcpf(d)));
            tm = fmaxf(tm, fabsf(m[c]));
            tv = fmaxf(tv, v[c]);
        }
        ms = row_scale(wave_max(tm), 1.0f / kMost4);
        vs = row_scale(wave_max(tv), 1.0f / kMost5);
        const float mi = ms > 0.0f ? reciprocal(ms) : 0.0f;
        const float vi = vs > 0.0f ? reciprocal(vs) : 0.0f;
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(m[0] * mi, m[1] * mi, 0, false);
        q.m.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(m[2] * mi, m[3] * mi, w, true);
        q.v.x = round_e5m2(v, vi, key, lane);
    }
}

// A tile's gradients at any element offset.  16-bit: aligned 8-byte words from
// the one that holds the tile's first element; with the tile ms elements into
// it, a quad is the upper part of its lane's word and the lower part of the
// next lane's (the next row's first word for lane 63; one more word after the
// last row).  Every word read holds an element of the tile, so none leaves the
// memory the tensor lies in.  fp32: quads of 4-byte alignment.
template <int GT, int R>
struct GradTile {
    v4f f[GT == ZERO_F32 ? R : 1];
    v2u w[GT == ZERO_F32 ? 1 : R + 1];
    int ms;
    __device__ __forceinline__ void load(const void* g, int lane) {
        if constexpr (GT == ZERO_F32) {
#pragma unroll
            for (int u = 0; u < R; ++u)
                f[u] = ldnt<v4f_a4>(static_cast<const float*>(g) + u * kRow + 4 * lane);
        } else {
            const uintptr_t at = (uintptr_t)g;
            ms = __builtin_amdgcn_readfirstlane((int)(at >> 1) & 3);
            const char* base = reinterpret_cast<const char*>(at & ~(uintptr_t)7);
#pragma unroll
            for (int u = 0; u < R; ++u) w[u] = ldnt<v2u>(base + u * 2 * kRow + 8 * lane);
            if (ms) w[R] = *reinterpret_cast<const v2u*>(base + R * 2 * kRow);
        }
    }
    __device__ __forceinline__ void quad(int u, float out[4]) const {
        if constexpr (GT == ZERO_F32) {
            out[0] = f[u].x; out[1] = f[u].y; out[2] = f[u].z; out[3] = f[u].w;
        } else {
            uint32_t lo = w[u].x, hi = w[u].y;
            if (ms) {
                const uint32_t nlo = from_above(lo, lane_value(w[u + 1].x, 0));
                const uint32_t nhi = from_above(hi, lane_value(w[u + 1].y, 0));
                const uint64_t x = ((uint64_t)hi << 32 | lo) >> (16 * ms) |
                                   ((uint64_t)nhi << 32 | nlo) << (64 - 16 * ms);
                lo = (uint32_t)x;
                hi = (uint32_t)(x >> 32);
            }
            out[0] = cvt16<GT>(lo & 0xffffu);
            out[1] = cvt16<GT>(lo >> 16);
            out[2] = cvt16<GT>(hi & 0xffffu);
            out[3] = cvt16<GT>(hi >> 16);
        }
    }
};

// A full tile's 16-bit parameters at any element offset: whole aligned words,
// each joined from a lane's values and the top of the lane below; the words
// shared with the tiles before and after are written element by element.
// KEEP: by plain stores, which leave the copy in the memory-side cache for the
// forward pass that reads it.
template <int R, bool KEEP>
struct CopyTile {
    uint16_t* lp;
    int ms;
    uint32_t carry_lo, carry_hi;
    __device__ __forceinline__ explicit CopyTile(uint16_t* at)
        : lp(at), ms((int)((uintptr_t)at >> 1) & 3), carry_lo(0), carry_hi(0) {}
    __device__ __forceinline__ static void put(uint16_t* p, v2u x) {
        if constexpr (KEEP) *reinterpret_cast<v2u*>(p) = x;
        else stnt<v2u>(p, x);
    }
    __device__ __forceinline__ void store(int u, const uint32_t h[4], int lane) {
        const int e = u * kRow + 4 * lane;
        const uint32_t lo = h[0] | h[1] << 16, hi = h[2] | h[3] << 16;
        if (ms == 0) {
            put(lp + e, v2u{lo, hi});
            return;
        }
        const uint32_t blo = from_below(lo, carry_lo), bhi = from_below(hi, carry_hi);
        const uint64_t x = ((uint64_t)hi << 32 | lo) << (16 * ms) |
                           ((uint64_t)bhi << 32 | blo) >> (64 - 16 * ms);
        carry_lo = lane_value(lo, 63);
        carry_hi = lane_value(hi, 63);
        if (u == 0 && lane == 0) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < 4 - ms) lp[c] = (uint16_t)h[c];
        } else {
            put(lp + e - ms, v2u{(uint32_t)x, (uint32_t)(x >> 32)});
        }
        if (u == R - 1 && lane == 63) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c >= 4 - ms) lp[e + c] = (uint16_t)h[c];
        }
    }
};

// Where a tile of R rows lies.
template <int GT, int R>
struct Place {
    const ZF_CONST MultiEntry* e;
    const char* g;
    uint16_t* lp;
    int64_t row, left;   // first arena row, elements from the tile's first on
    __device__ __forceinline__ Place(const MultiAdamLaunch& a, int tile) {
        e = as_const(a.entries) + as_const(a.tile_tensor)[tile];
        const int64_t row_in = (int64_t)(tile - e->tile0) * R;
        const int64_t at = row_in * kRow;
        row = e->row0 + row_in;
        left = e->numel - at;
        g = static_cast<const char*>(e->grad) + at * (GT == ZERO_F32 ? 4 : 2);
        lp = static_cast<uint16_t*>(e->param) + at;
    }
    __device__ __forceinline__ bool whole() const { return left >= R * kRow; }
};

// A tile on its way: load() issues every load, update() waits for them.  Rows
// of the tile are WHOLE, or end after p.left elements (a tensor's last tile):
// then gradient and copy go element-wise.
template <int GT, int PT, int BITS, int R, bool WHOLE, bool KEEP>
struct Tile {
    GradTile<GT, R> gt;
    uint32_t ge[WHOLE ? 1 : R][4];   // gradient elements as stored
    Quad<BITS> q[R];
    uint32_t scales;                 // lane u: the m scale of row u, lane R + u: its v scale

    __device__ __forceinline__ static int rows(const Place<GT, R>& p) {
        return WHOLE ? R : (int)((p.left + kRow - 1) / kRow);
    }
    __device__ __forceinline__ void load(const MultiAdamLaunch& a, const Place<GT, R>& p, int lane) {
        if constexpr (WHOLE) gt.load(p.g, lane);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (!WHOLE && u * kRow >= p.left) break;
            load_state<BITS>(a, (p.row + u) * kRow + 4 * lane, q[u]);
            if constexpr (!WHOLE) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int i = u * kRow + 4 * lane + c;
                    ge[u][c] = 0;
                    if (i < p.left) {
                        if constexpr (GT == ZERO_F32) ge[u][c] = reinterpret_cast<const uint32_t*>(p.g)[i];
                        else ge[u][c] = reinterpret_cast<const uint16_t*>(p.g)[i];
                    }
                }
            }
        }
        if constexpr (BITS == 8) {
            const int n = rows(p), r = lane < R ? lane : lane - R;
            scales = 0;
            if (r < n) scales = __float_as_uint((lane < R ? a.ms : a.vs)[p.row + r]);
        }
    }
    __device__ __forceinline__ void update(const MultiAdamLaunch& a, const MultiScalars& s,
                                           const Place<GT, R>& p, int lane) {
        if (s.skip) return;
        const TensorScalars t = tensor_scalars<BITS>(s, p.e);
        CopyTile<R, KEEP> copy(p.lp);
        uint32_t out = 0;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (!WHOLE && u * kRow >= p.left) break;
            float gv[4];
            if constexpr (WHOLE) {
                gt.quad(u, gv);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    gv[c] = GT == ZERO_F32 ? __uint_as_float(ge[u][c]) : cvt16<GT>(ge[u][c]);
            }
            float ms = 0.0f, vs = 0.0f;
            uint32_t key = 0;
            if constexpr (BITS == 8) {
                ms = __uint_as_float(lane_value(scales, u));
                vs = __uint_as_float(lane_value(scales, R + u));
                key = mix(s.key + (uint32_t)(p.row + u));
            }
            update_quad<BITS>(a, s, t, gv, q[u], ms, vs, key, lane);
            store_state<BITS>(a, (p.row + u) * kRow + 4 * lane, q[u]);
            if constexpr (PT != ZERO_NONE) {
                uint32_t h[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) h[c] = round16<PT>(q[u].p[c]);
                if constexpr (WHOLE) {
                    copy.store(u, h, lane);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int i = u * kRow + 4 * lane + c;
                        if (i < p.left) p.lp[i] = (uint16_t)h[c];
                    }
                }
            }
            if constexpr (BITS == 8) {
                if (lane == u) out = __float_as_uint(ms);
                if (lane == R + u) out = __float_as_uint(vs);
            }
        }
        if constexpr (BITS == 8) {
            const int n = rows(p), r = lane < R ? lane : lane - R;
            if (r < n) (lane < R ? a.ms : a.vs)[p.row + r] = __uint_as_float(out);
        }
    }
};

// One wave per tile, in launches of at most kSliceTiles tiles over consecutive
// ranges, with at most two blocks per compute unit for 32-bit states and four
// for 8-bit ones, which have half the bytes in flight per wave (a dynamic LDS
// reservation that the kernel does not use): both keep the addresses in flight
// in one window of every array.  One launch against slices (no limit), us:
// 1.25e9 elements with 8-bit states 3941 and 3633, 2.02e8 and 3e7 within 1%.
// Whole steps over slices, in turn on three allocations (medians, us):
//   blocks per CU             no limit      4        3        2
//   2.02e8, 32-bit              1004      1007     1004      982
//   1e8, 32-bit                  487       490      484      484
//   3e7, 32-bit                  142       139      137      137
//   2.5e7, 32-bit                132       132      132      133
//   2.02e8, 8-bit                572       573      565      582
//   1e8, 8-bit                   294       290      294      307
//   3e7, 8-bit                    81        79       81       87
//   2.5e7, 8-bit, no copy         82.5      84       88       84
//   1.25e9, 8-bit               3660      3648     3594     3578
// Two for 32-bit states is the best or within 1% of it; four for 8-bit ones is
// within 2% of the best on every line, which no other is.  Slices of half and
// twice the size are within 2%.  A resident grid taking
// tiles from a counter in the order its blocks ask (the flat step's form for
// large shards) took 1008 against 1016 us on the first line's list, 613
// against 604 on the third's and 162 against 147 on the second's (before
// gradients were kept).
constexpr int kSliceTiles = 131072;
// A copy of at most this size, counted in whole tiles, is left in the memory-side
// cache (KEEP).  Steps
// without and with, us: 3e7 elements 151 and 138 (32-bit states), 87 and 79
// (8-bit); 1e8 503 and 445, 280 and 243; with statistics, whose kept gradients
// compete for the cache, 518 and 486, 294 and 289, but 1.3e8 674 and 655, 379
// and 386, and 2.02e8 1000 and 1034, 572 and 624.
constexpr int64_t kKeepCopyBytes = (int64_t)192 << 20;
constexpr unsigned kLdsTwoBlocks = 56 * 1024, kLdsFourBlocks = 40 * 1024;
template <int GT, int PT, int BITS, int R, bool KEEP>
__global__ void __launch_bounds__(kThreads) multi_adamw_kernel(MultiAdamLaunch a, int tile0) {
    const int lane = threadIdx.x & 63;
    const int tile = tile0 + (int)blockIdx.x * kWaves +
                     __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (tile >= a.n_tiles) return;
    const MultiScalars s = load_record(a.scalars);
    const Place<GT, R> p(a, tile);
    if (p.whole()) {
        Tile<GT, PT, BITS, R, true, KEEP> t;
        t.load(a, p, lane);
        t.update(a, s, p, lane);
    } else {
        Tile<GT, PT, BITS, R, false, KEEP> t;
        t.load(a, p, lane);
        t.update(a, s, p, lane);
    }
}

// A short list's update with statistics, the second of two launches: every
// block folds the spans' sums itself while its tile is on the way, forms the
// step's scalars, and updates.  The first sum_blocks blocks have no tiles:
// block 0 writes the state, which the others read from the copy that the
// statistics pass took, and each of their waves adds one tensor's sums.  Saves
// the fold's launch and its time, 2.8 us of the small MLP's 13.4; every block
// reads all partial sums, so a list of more than kMultiShortSpans spans takes
// the fold.
static_assert(kMultiShortSpans % kThreads == 0, "whole partial sums per thread");
template <int GT, int PT, int BITS, int R>
__global__ void __launch_bounds__(kThreads) multi_adamw_short_kernel(MultiAdamLaunch a,
                                                                     MultiNormLaunch n,
                                                                     MultiStep step,
                                                                     int sum_blocks) {
    __shared__ double sums[kWaves];
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    constexpr int kMine = (int)(kMultiShortSpans / kThreads);   // partial sums per thread
    double part[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
        const int i = threadIdx.x + j * kThreads;
        part[j] = i < n.n_spans ? n.partials[i] : 0.0;
    }
    const int tile = ((int)blockIdx.x - sum_blocks) * kWaves + w;
    const bool live = tile >= 0 && tile < a.n_tiles;
    const Place<GT, R> p(a, live ? tile : 0);
    const bool whole = live && p.whole();
    Tile<GT, PT, BITS, R, true, true> t;
    Tile<GT, PT, BITS, R, false, true> tp;
    if (whole) t.load(a, p, lane);
    else if (live) tp.load(a, p, lane);
    double x = part[0];
#pragma unroll
    for (int j = 1; j < kMine; ++j) x += part[j];
    x = wave_sum(x);
    if (lane == 0) sums[w] = x;
    __syncthreads();
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < kWaves; ++j) total += sums[j];
    MultiState st = load_record(n.snapshot);
    add_sum(st, total, 0);
    const MultiScalars s = step_scalars(step, st);
    if (whole) t.update(a, s, p, lane);
    else if (live) tp.update(a, s, p, lane);
    if (tile >= 0) return;
    if (blockIdx.x == 0 && threadIdx.x == 0) write_state(step, st, s);
    const int k = (int)blockIdx.x * kWaves + w;
    if (k >= n.n_tensors) return;
    const int p0 = as_const(a.entries)[k].span0, np = as_const(a.entries)[k].n_spans;
    double z = 0.0;
    for (int i = lane; i < np; i += 64) z += n.partials[p0 + i];
    z = wave_sum(z);
    if (lane == 0) n.tensor_sumsq[k] = z;
}

// A launch by the runtime's plain entry point, 0.15 us less of the host's time
// than the launch syntax, which passes the shape through a second call.
template <typename... P, typename... A>
int launch(void (*kernel)(P...), unsigned grid, unsigned block, unsigned lds, hipStream_t s,
           const A&... args) {
    static_assert((std::is_same<P, A>::value && ...), "arguments of the kernel's own types");
    void* p[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    const int e = (int)hipLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(block),
                                       p, lds, s);
    if (e) (void)hipGetLastError();   // reported here, not by the next call
    return e;
}

// n, step: for multi_adamw_short_kernel, or null
template <int GT, int PT, int BITS, int R>
int launch_short(const MultiAdamLaunch& a, const MultiNormLaunch* n, const MultiStep* step,
                 hipStream_t s) {
    const int tile_blocks = (a.n_tiles + kWaves - 1) / kWaves;
    if (!n)
        return launch(multi_adamw_kernel<GT, PT, BITS, R, true>, (unsigned)tile_blocks, kThreads, 0, s,
                      a, 0);
    const int sum_blocks = (n->n_tensors + kWaves - 1) / kWaves;
    return launch(multi_adamw_short_kernel<GT, PT, BITS, R>, (unsigned)(sum_blocks + tile_blocks),
                  kThreads, 0, s, a, *n, *step, sum_blocks);
}
template <int GT, int PT, int BITS, bool KEEP>
int launch_long(const MultiAdamLaunch& a, hipStream_t s) {
    for (int t0 = 0; t0 < a.n_tiles; t0 += kSliceTiles) {
        const int tiles = a.n_tiles - t0 < kSliceTiles ? a.n_tiles - t0 : kSliceTiles;
        const int e = launch(multi_adamw_kernel<GT, PT, BITS, kMultiRowsLong, KEEP>,
                             (unsigned)((tiles + kWaves - 1) / kWaves), kThreads,
                             BITS == 32 ? kLdsTwoBlocks : kLdsFourBlocks, s, a, t0);
        if (e) return e;
    }
    return 0;
}
template <int GT, int PT, int BITS>
int launch_update(const MultiAdamLaunch& a, const MultiNormLaunch* n, const MultiStep* step,
                  hipStream_t s) {
    if (a.n_tiles == 0) return 0;
    if (a.tile_rows == kMultiRowsTiny)
        return launch_short<GT, PT, BITS, kMultiRowsTiny>(a, n, step, s);
    if (a.tile_rows == kMultiRowsShort)
        return launch_short<GT, PT, BITS, kMultiRowsShort>(a, n, step, s);
    if constexpr (PT != ZERO_NONE) {
        const int64_t copy_bytes = (int64_t)a.n_tiles * kMultiRowsLong * kRow * 2;
        if (copy_bytes <= kKeepCopyBytes) return launch_long<GT, PT, BITS, true>(a, s);
    }
    return launch_long<GT, PT, BITS, false>(a, s);
}
template <int GT, int PT>
int launch_update(const MultiAdamLaunch& a, const MultiNormLaunch* n, const MultiStep* p, hipStream_t s) {
    return a.bits == 8 ? launch_update<GT, PT, 8>(a, n, p, s) : launch_update<GT, PT, 32>(a, n, p, s);
}
template <int GT>
int launch_update(const MultiAdamLaunch& a, const MultiNormLaunch* n, const MultiStep* p, hipStream_t s) {
    if (a.pdtype == ZERO_F16) return launch_update<GT, ZERO_F16>(a, n, p, s);
    if (a.pdtype == ZERO_BF16) return launch_update<GT, ZERO_BF16>(a, n, p, s);
    return launch_update<GT, ZERO_NONE>(a, n, p, s);
}
int launch_update(const MultiAdamLaunch& a, const MultiNormLaunch* n, const MultiStep* p, hipStream_t s) {
    if (a.gdtype == ZERO_F32) return launch_update<ZERO_F32>(a, n, p, s);
    if (a.gdtype == ZERO_F16) return launch_update<ZERO_F16>(a, n, p, s);
    return launch_update<ZERO_BF16>(a, n, p, s);
}

int launch_stats(const MultiNormLaunch& a, hipStream_t s) {
    if (a.n_spans == 0) return 0;
    const unsigned grid = (unsigned)a.n_spans;
    if (a.dtype == ZERO_F32) return launch(multi_stats_kernel<ZERO_F32>, grid, kThreads, 0, s, a);
    if (a.dtype == ZERO_F16) return launch(multi_stats_kernel<ZERO_F16>, grid, kThreads, 0, s, a);
    return launch(multi_stats_kernel<ZERO_BF16>, grid, kThreads, 0, s, a);
}
int launch_fold(const MultiNormLaunch& a, const MultiStep* step, hipStream_t s) {
    // a wave per tensor where the tensors have few spans each on average
    const int per_wave = a.n_spans <= 64 * (int64_t)a.n_tensors;
    const unsigned per = per_wave ? kFoldThreads / 64 : 1;
    const unsigned grid = 1 + ((unsigned)a.n_tensors + per - 1) / per;
    return step ? launch(multi_fold_step_kernel, grid, kFoldThreads, 0, s, a, *step, per_wave)
                : launch(multi_fold_kernel, grid, kFoldThreads, 0, s, a, per_wave);
}

}  // namespace

int launch_multi_norm(const MultiNormLaunch& a, void* stream) {
    if (const int e = launch_stats(a, (hipStream_t)stream)) return e;
    return launch_fold(a, nullptr, (hipStream_t)stream);
}

int launch_multi_step(const MultiAdamLaunch& a, const MultiNormLaunch* norm, const MultiStep& step,
                      void* stream) {
    hipStream_t s = (hipStream_t)stream;
    if (!norm) {
        if (const int e = launch(multi_prepare_kernel, 1, 64, 0, s, step)) return e;
        return launch_update(a, nullptr, nullptr, s);
    }
    MultiNormLaunch n = *norm;
    const int64_t keep = kKeepBytes / (n.span * (n.dtype == ZERO_F32 ? 4 : 2));
    n.keep_spans = keep < n.n_spans ? (int32_t)keep : n.n_spans;
    const bool fold_in_update = a.tile_rows != kMultiRowsLong && a.n_tiles > 0;
    if (!fold_in_update) n.snapshot = nullptr;
    if (const int e = launch_stats(n, s)) return e;
    if (fold_in_update) return launch_update(a, &n, &step, s);
    if (const int e = launch_fold(n, &step, s)) return e;
    return launch_update(a, nullptr, nullptr, s);
}

}  // namespace zf
