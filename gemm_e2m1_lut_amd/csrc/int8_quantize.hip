// int8_quantize.hip -- rows of bf16 or fp32 values to int8 codes with one fp32
// scale per row: int8_quantize, rmsnorm_int8_quantize, silu_mul_int8_quantize
// (the left operands of int8_gemm, and its weights per output channel).
//
// Mathematics. A row of values p_c gives pmax = max |p_c|, codes q_c = the
// integer nearest to 127 p_c / pmax (ties to even) and a scale s with
// p_c ~ s q_c, where p is
//   plain   x                          s = pmax / 127
//   norm    fl32(h w), h = fl32(x + r) s = pmax / (127 sqrt(mean(h^2) + eps))
//   act     silu(gate) up              s = pmax / 127
// The norm's factor 1 / sqrt(mean(h^2) + eps) is the same for the whole row, so
// it cancels in the codes and enters only the scale: one reduction carries
// both the largest magnitude and the sum of squares, and the codes do not
// depend on how that sum is rounded. The sum is kept in 64 bits: the squares of
// every finite fp32 fit, and no partial sum loses what the fp32 scale shows.
//
// Codes are decided on the exact quotient. v = fl32(p fl32(127 / pmax)) is
// within 127 * 2^-23 < 2^-15 of 127 p / pmax; where v lies further than
// kNear = 2^-14 from a half-integer, rounding v gives the code. Otherwise
// (about one element in 8000) the sign of 254 p - (2 j + 1) pmax decides,
// which one fp64 fma gives without error (254 p and (2 j + 1) pmax have at
// most 32 bits). Outside 2^-100 <= pmax <= 2^100 the row is first multiplied by
// 2^64 or 2^-64, so that neither 127 / pmax nor a product leaves the fp32
// range; elements that this flushes are below half a code.
// silu(gate) up is not an fp32 number. Its fp32 evaluation is within 9.4 * 2^-24
// of it (relatively; the sum of the roundings of the exponent, of exp2, of 1 +
// e^-a, of the reciprocal, one ulp each for the hardware's, and of three
// products), so the largest magnitude is taken in fp64 over the elements within
// 2^-18 of the largest fp32 value, and codes whose v (then within 127 * 12.4 *
// 2^-24 < 1.54 * 2^-14) is within kNearAct of a half-integer are decided in fp64
// (one element in 5000).
//
// The largest magnitude is an integer maximum of the magnitude patterns: a NaN
// has the largest pattern, so a row that holds a NaN or an infinity (or whose
// product overflows) shows at once; it gets the scale NaN and codes 0.
//
// gfx950 design. All three stream memory: 3 bytes an element (plain, bf16), 7
// (norm with residual), 5 (act). A row is held in registers between the
// reduction and the codes, so every input is read once (rows of more than
// 16384 columns are read again for the codes); a thread takes units of 8 columns
// (16-byte loads, 8-byte stores), all of its loads are issued before the first
// is used. Measured: plain 14336 x 4096 32.1 us (5.5 TB/s), norm with residual
// 8192 x 4096 43.5 us (5.4 TB/s), both what a copy with that mix of reads and
// writes takes; act 2048 x 14336 32.5 us (4.5 TB/s; its fp64 decisions wait for
// their two values from memory again).
#include "device.hpp"
#include "kernels.hpp"

namespace e2m1 {
namespace {

enum Op { kPlain, kNorm, kNormRes, kAct };

constexpr float kNear = 0x1p-14f;
constexpr float kNearAct = 0x1.ap-14f;
constexpr uint32_t kInfBits = 0x7F800000u;

// ------------------------------------------------------------ reductions --

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
}

template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp_u32<kCtrl>((uint32_t)u) |
                                          ((uint64_t)dpp_u32<kCtrl>((uint32_t)(u >> 32)) << 32));
}

__device__ __forceinline__ double shfl_f64(double v, int mask) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __shfl_xor((uint32_t)u, mask, kWave), hi = __shfl_xor((uint32_t)(u >> 32), mask, kWave);
    return __builtin_bit_cast(double, (uint64_t)lo | ((uint64_t)hi << 32));
}

// Every lane ends with the wave's maximum / sum / maximum.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));
    v = max(v, dpp_u32<0x4E>(v));
    v = max(v, dpp_u32<0x141>(v));
    v = max(v, dpp_u32<0x140>(v));
    v = max(v, (uint32_t)__shfl_xor(v, 16, kWave));
    return max(v, (uint32_t)__shfl_xor(v, 32, kWave));
}

__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    v += shfl_f64(v, 16);
    return v + shfl_f64(v, 32);
}

__device__ __forceinline__ double wave_max_f64(double v) {
    v = fmax(v, dpp_f64<0xB1>(v));
    v = fmax(v, dpp_f64<0x4E>(v));
    v = fmax(v, dpp_f64<0x141>(v));
    v = fmax(v, dpp_f64<0x140>(v));
    v = fmax(v, shfl_f64(v, 16));
    return fmax(v, shfl_f64(v, 32));
}

// ------------------------------------------------------------------- load --

template <typename T>
struct Unit;   // eight values as loaded

template <>
struct Unit<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ void put(uint16_t* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    static __device__ __forceinline__ double one(const uint16_t* p) {
        return (double)__uint_as_float((uint32_t)*p << 16);
    }
};

template <>
struct Unit<float> {
    f32x4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *reinterpret_cast<const f32x4*>(p);
        b = *reinterpret_cast<const f32x4*>(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    }
    static __device__ __forceinline__ void put(float* p, const float (&v)[8]) {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
    static __device__ __forceinline__ double one(const float* p) { return (double)*p; }
};

// -------------------------------------------------------------------- act --

// silu(g) u in fp32, within 2^-20 of the exact value relatively wherever that
// is 2^-110 or more: with a = |g|, e^-a = w 2^t, t = ceil(1/2 - a log2 e)
// and w in (0.35, 0.71], it is u g / (1 + e^-a) for g >= 0 and u w 2^t g / (1 + e^-a)
// for g < 0. The power of two joins u last, so neither a very negative gate nor
// a large `up` overflows on the way. The exponent's argument takes two words of
// log2 e (16 bits and the rest for a bf16 gate, 24 for an fp32 one), each in an
// fma: the first one's product joins t unrounded, whose own rounding (as the
// argument of ceil) only moves the border between two values of t. (That border
// is kept off w = 1, past which u w could overflow.) a is capped at 1000
// (e^-1000 times any fp32 is 0 in fp32); the factor g keeps NaN and infinity.
template <bool kBf16>
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float a = fminf(fabsf(g), 1000.f);
    float t, e;   // the exponent of 2 is t + e
    if constexpr (kBf16) {
        t = ceilf(fmaf(a, -0x1.7154p+0f, 0.5f));
        e = fmaf(a, -0x1.d94ae0p-18f, fmaf(a, -0x1.7154p+0f, -t));
    } else {
        t = ceilf(fmaf(a, -0x1.715476p+0f, 0.5f));
        e = fmaf(a, -0x1.4ae0cp-26f, fmaf(a, -0x1.715476p+0f, -t));
    }
    const float w = __builtin_amdgcn_exp2f(e);
    const int ti = (int)t;
    const float r = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_ldexpf(w, ti));
    const float n = g < 0.f ? __builtin_amdgcn_ldexpf(u * w, ti) : u;
    return n * r * g;   // (n g could overflow where the result does not)
}

// The same for |g| <= kNearGate (or NaN), in half the instructions (act 2048 x 14336: 36.2 -> 32.5 us): e^-g =
// 2^t (1 + x), t = fl32(-g log2 e) and x the rest of the exponent times ln 2 (bf16: t is exact, x is the second word's
// part, at most 2.2e-4). 2^t is at most 2^64, so no power of two has to be kept apart. Errors, in 2^-24: 0.4 of
// x^2 / 2, 1 each of 1 + x, of the sum and of two products, 2 each of 2^t and the reciprocal: 8.4. u / (1 + e^-g) is
// subnormal only where the result is below 2^-120, whose code is 0 in every row that is not taken in fp64.
constexpr float kNearGate = 44.f;

template <bool kBf16>
__device__ __forceinline__ float silu_mul_near(float g, float u) {
    float t, f;
    if constexpr (kBf16) {
        t = g * -0x1.7154p+0f;
        f = fmaf(g, -0x1.480fb4p-18f, 1.f);
    } else {
        t = g * -0x1.715476p+0f;
        f = fmaf(fmaf(g, -0x1.4ae0cp-26f, fmaf(g, -0x1.715476p+0f, -t)), 0x1.62e430p-1f, 1.f);
    }
    return u * __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(t), f, 1.f)) * g;
}

__device__ __forceinline__ double silu_mul_f64(double g, double u) { return g / (1.0 + exp(-g)) * u; }

// ------------------------------------------------------------------ codes --

// Code of p (magnitude at most pm, both multiplied by the row's power of two):
// nearest integer to 127 p / pm, ties to even, from v close to that quotient.
__device__ __forceinline__ int exact_code(float p, double pm, float v) {
    const int j = (int)fabsf(v);
    const double d = fma(254.0, (double)fabsf(p), -((double)(2 * j + 1) * pm));   // its sign is exact
    const int q = d > 0.0 ? j + 1 : d < 0.0 ? j : j + (j & 1);
    return p < 0.f ? -q : q;
}

constexpr float kMagic = 12582912.f;   // 1.5 * 2^23: v + kMagic holds rint(v) in its low bits

// Threads of a workgroup: one row, or four of one wave each.
constexpr int rows_block(int threads_per_row) { return threads_per_row == kWave ? 4 * kWave : threads_per_row; }

template <typename T, int kOp, int kTpr, int kUnits, bool kLong>
__global__ __launch_bounds__(rows_block(kTpr)) void int8_rows_kernel(
    const T* __restrict__ x, const T* residual, const T* __restrict__ weight, float eps, T* residual_out,
    int8_t* __restrict__ q, float* __restrict__ scale, int64_t rows, int k) {
    constexpr int kRowsPerBlock = rows_block(kTpr) / kTpr;
    constexpr int kWaves = kTpr / kWave;
    constexpr bool kIsNorm = kOp == kNorm || kOp == kNormRes;
    static_assert(kTpr % kWave == 0, "whole waves");
    const int t = kRowsPerBlock > 1 ? threadIdx.x % kTpr : threadIdx.x;
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t row = block * kRowsPerBlock + (kRowsPerBlock > 1 ? threadIdx.x / kTpr : 0);
    if (row >= rows) return;   // whole waves, or the whole workgroup where it has barriers
    const int units = k / 8;
    const T* xr = x + row * (kOp == kAct ? 2 * (int64_t)k : k);
    const T* rr = kOp == kNormRes ? residual + row * (int64_t)k : nullptr;
    T* hr = kOp == kNormRes ? residual_out + row * (int64_t)k : nullptr;
    int8_t* qr = q + row * (int64_t)k;

    float p[kUnits][8];
    // largest patterns with the sign bit (as unsigned numbers: the largest magnitude among the negative values, NaN
    // above all) and without (as signed numbers: among the others)
    uint32_t mneg = 0;
    int32_t mpos = 0;
    double ss = 0.0;       // sum of squares of h
    constexpr int span = kTpr * kUnits;   // units a pass of the threads covers

    // p of the units base + t, base + t + kTpr, ... A thread past the row's end repeats the row's last unit (which
    // changes no maximum) and stores nothing; with a residual, whose last unit may be overwritten by then, its p are 0.
    auto fetch = [&](int base, bool first) __attribute__((always_inline)) {
        Unit<T> a[kUnits], b[kUnits], c[kUnits];
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            if (j > 0 && base + j * kTpr >= units) continue;   // uniform: the whole pass is past the end
            const int at = 8 * min(base + t + j * kTpr, units - 1);
            a[j].load(xr + at);
            if constexpr (kOp == kAct) b[j].load(xr + k + at);
            if constexpr (kOp == kNormRes) b[j].load(rr + at);
            if constexpr (kIsNorm) c[j].load(weight + at);
        }
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            if (j > 0 && base + j * kTpr >= units) continue;
            const int u = base + t + j * kTpr;
            const bool live = u < units;
            float va[8], vb[8], vc[8];
            a[j].get(va);
            if constexpr (kOp == kAct || kOp == kNormRes) b[j].get(vb);
            if constexpr (kIsNorm) c[j].get(vc);
            if constexpr (kOp == kNormRes) {
#pragma unroll
                for (int i = 0; i < 8; ++i) va[i] += vb[i];
                // each thread writes only what it has read, so residual_out may be residual;
                // a long row reads it twice and writes on the second pass
                if (live && first != kLong) Unit<T>::put(hr + 8 * u, va);
            }
            if constexpr (kOp == kAct) {
                float gate = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) gate = fmaxf(gate, fabsf(va[i]));
                if (gate <= kNearGate) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[j][i] = silu_mul_near<sizeof(T) == 2>(va[i], vb[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[j][i] = silu_mul<sizeof(T) == 2>(va[i], vb[i]);
                }
            }
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (kOp != kAct) p[j][i] = kIsNorm ? va[i] * vc[i] : va[i];
                if constexpr (kOp == kNormRes) p[j][i] = live ? p[j][i] : 0.f;
                if constexpr (kIsNorm) s = fma((double)va[i], (double)va[i], s);
                if (first) {
                    mneg = max(mneg, __float_as_uint(p[j][i]));
                    mpos = max(mpos, __float_as_int(p[j][i]));
                }
            }
            if constexpr (kIsNorm) {
                if (first && live) ss += s;
            }
        }
    };

    if constexpr (kLong) {
        for (int base = 0; base < units; base += span) fetch(base, true);
    } else {
        fetch(0, true);
    }

    // the thread's largest magnitude pattern, then the row's
    const uint32_t mine = max(mneg > 0x7FFFFFFFu ? mneg & 0x7FFFFFFFu : 0u, (uint32_t)mpos);
    uint32_t m = wave_max_u32(mine);
    if constexpr (kIsNorm) ss = wave_sum_f64(ss);
    if constexpr (kWaves > 1) {
        __shared__ uint32_t wm[kWaves];
        __shared__ double wss[kIsNorm ? kWaves : 1];
        const int lane = t % kWave;
        if (lane == 0) {
            wm[t / kWave] = m;
            if constexpr (kIsNorm) wss[t / kWave] = ss;
        }
        __syncthreads();
        m = wm[lane % kWaves];
#pragma unroll
        for (int d = kWaves / 2; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor(m, d, kWave));
        if constexpr (kIsNorm) {
            ss = wss[lane % kWaves];
#pragma unroll
            for (int d = kWaves / 2; d > 0; d >>= 1) ss += shfl_f64(ss, d);
        }
    }

    // row-uniform from here on
    const float top = __uint_as_float(m);
    if (m >= kInfBits || m == 0) {   // non-finite, or all zero
        if constexpr (kOp == kNormRes && kLong)   // h is still to be written
            for (int base = 0; base < units; base += span) fetch(base, false);
        for (int u = t; u < units; u += kTpr) *reinterpret_cast<uint2*>(qr + 8 * u) = make_uint2(0u, 0u);
        if (t == 0) scale[row] = m == 0 ? 0.f : __uint_as_float(0x7FC00000u);
        return;
    }
    // rows outside the range where fl32 steps are safe are multiplied by a power of two first
    const float pre = top > 0x1p100f ? 0x1p-64f : top < 0x1p-100f ? 0x1p64f : 1.f;

    // act: the largest magnitude in fp64, over the elements whose fp32 value is near the largest
    double pm = (double)(top * pre);
    double pm_act = 0.0;
    const bool tiny = kOp == kAct && top < 0x1p-60f;   // fp32 values may be subnormal: every element in fp64
    // |silu(gate) up| of the unit's elements whose bit is set in mask
    auto largest = [&](int u, uint32_t mask) __attribute__((always_inline)) {
        while (mask != 0) {
            const int c = 8 * u + __builtin_ctz(mask);
            mask &= mask - 1;
            pm_act = fmax(pm_act, fabs(silu_mul_f64(Unit<T>::one(xr + c), Unit<T>::one(xr + k + c))));
        }
    };
    if constexpr (kOp == kAct) {
        const float near = tiny ? 0.f : top * (1.f - 0x1p-18f);
        auto scan = [&](int base) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < kUnits; ++j) {
                const int u = base + t + j * kTpr;
                if (u >= units) continue;
                uint32_t mask = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) mask |= (uint32_t)(fabsf(p[j][i]) >= near) << i;
                largest(u, mask);
            }
        };
        if (__uint_as_float(mine) >= near) {   // few threads have such an element
            if constexpr (kLong) {
                for (int base = 0; base < units; base += span) {
                    fetch(base, false);
                    scan(base);
                }
            } else {
                scan(0);
            }
        }
        pm_act = wave_max_f64(pm_act);
        if constexpr (kWaves > 1) {
            __shared__ double wp[kWaves];
            const int lane = t % kWave;
            if (lane == 0) wp[t / kWave] = pm_act;
            __syncthreads();
            pm_act = wp[lane % kWaves];
#pragma unroll
            for (int d = kWaves / 2; d > 0; d >>= 1) pm_act = fmax(pm_act, shfl_f64(pm_act, d));
        }
        pm = pm_act * (double)pre;
    }

    if (t == 0) {
        double s;
        if constexpr (kOp == kAct) s = pm_act / 127.0;
        else if constexpr (kOp == kPlain) s = (double)top / 127.0;
        else s = (double)top / (127.0 * sqrt(ss / (double)k + (double)eps));
        scale[row] = (float)s;
    }

    const float inv = 127.f / (float)pm;
    auto codes = [&](int base) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int u = base + t + j * kTpr;
            if (u >= units) continue;
            if (pre != 1.f) {
#pragma unroll
                for (int i = 0; i < 8; ++i) p[j][i] *= pre;
            }
            uint32_t c[8];
            float off = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = p[j][i] * inv;
                const float z = v + kMagic;
                off = fmaxf(off, fabsf(v - (z - kMagic)));
                c[i] = __float_as_uint(z);
            }
            if constexpr (kOp != kAct) {
                if (off > 0.5f - kNear) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) c[i] = (uint32_t)exact_code(p[j][i], pm, p[j][i] * inv);
                }
            }
            // the low bytes of four words each
            const uint32_t lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0C0C0400u),
                                                      __builtin_amdgcn_perm(c[1], c[0], 0x0C0C0400u), 0x05040100u);
            const uint32_t hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[7], c[6], 0x0C0C0400u),
                                                      __builtin_amdgcn_perm(c[5], c[4], 0x0C0C0400u), 0x05040100u);
            *reinterpret_cast<uint2*>(qr + 8 * u) = make_uint2(lo, hi);
            if constexpr (kOp == kAct) {
                if (off > 0.5f - kNearAct || tiny) {   // codes near a border: the byte is written again
                    uint32_t mask = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float v = p[j][i] * inv;
                        mask |= (uint32_t)(fabsf(v - rintf(v)) > 0.5f - kNearAct || tiny) << i;
                    }
                    while (mask != 0) {
                        const int e = 8 * u + __builtin_ctz(mask);
                        mask &= mask - 1;
                        const double P = silu_mul_f64(Unit<T>::one(xr + e), Unit<T>::one(xr + k + e));
                        qr[e] = (int8_t)(int)rint(P * 127.0 / pm_act);
                    }
                }
            }
        }
    };
    if constexpr (kLong) {
        for (int base = 0; base < units; base += span) {
            fetch(base, false);
            codes(base);
        }
    } else {
        codes(0);
    }
}

constexpr int64_t kGridX = 1 << 20;   // times 1024 threads: below the 2^32 of a grid dimension

template <typename T, int kOp, int kTpr, int kUnits, bool kLong>
void launch_rows(const T* x, const T* residual, const T* weight, float eps, T* residual_out, int8_t* q, float* scale,
                 int64_t rows, int64_t k, hipStream_t stream) {
    constexpr int kRowsPerBlock = rows_block(kTpr) / kTpr;
    const int64_t blocks = (rows + kRowsPerBlock - 1) / kRowsPerBlock;
    const int64_t gx = blocks < kGridX ? blocks : kGridX;
    const dim3 grid((unsigned)gx, (unsigned)((blocks + gx - 1) / gx));
    int8_rows_kernel<T, kOp, kTpr, kUnits, kLong><<<grid, rows_block(kTpr), 0, stream>>>(
        x, residual, weight, eps, residual_out, q, scale, rows, (int)k);
}

template <typename T, int kOp>
hipError_t dispatch(const void* xv, const void* resv, const void* wv, float eps, void* outv, int8_t* q, float* scale,
                    int64_t rows, int64_t k, hipStream_t stream) {
    const T* x = static_cast<const T*>(xv);
    const T* r = static_cast<const T*>(resv);
    const T* w = static_cast<const T*>(wv);
    T* h = static_cast<T*>(outv);
    const int64_t units = k / 8;
#define E2M1_ROWS(TPR, UNITS, LONG) \
    launch_rows<T, kOp, TPR, UNITS, LONG>(x, r, w, eps, h, q, scale, rows, k, stream)
    // Few elements: as many threads a row as it has units, for the latency. Many: two units or more a thread, for the
    // bytes in flight. us in a graph, the one against the other, bf16:
    //   plain               1 x 4096 2.7 / 2.9, 128 x 1024 2.8 / 3.7, 1024 x 4096 5.1 / 5.0, 8192 x 4096 25.4 / 21.5
    //   norm with residual  1 x 4096 3.2 / 3.6, 128 x 4096 3.8 / 4.3, 2000 x 4096 13.0 / 12.7, 8192 x 8192 90.4 / 82.7
    //   act                 1 x 14336 4.9 / 5.3, 16 x 14336 5.6 / 6.1, 1024 x 8192 12.4 / 11.6, 8192 x 4096 37.5 / 32.8
    // fp32, whose units have twice the bytes: the same for few (plain 128 x 1024 2.7 / 2.9, act 16 x 14336 5.9 / 6.5),
    // and for many not enough on either side for a rule of its own (8192 x 4096: plain 30.6 / 31.1, norm 78.4 / 79.3,
    // act 53.1 / 57.6; 2000 x 8192: act 31.2 / 29.2).
    const bool many = rows * k >= (int64_t)6 << 20;
    if (units <= 64) {
        E2M1_ROWS(64, 1, false);
    } else if (units <= 128) {
        if (many) E2M1_ROWS(64, 2, false);
        else E2M1_ROWS(128, 1, false);
    } else if (units <= 256) {
        if (many) E2M1_ROWS(128, 2, false);
        else E2M1_ROWS(256, 1, false);
    } else if (units <= 512) {
        if (many) E2M1_ROWS(256, 2, false);
        else E2M1_ROWS(512, 1, false);
    } else if (units <= 1024) {
        if (many) E2M1_ROWS(512, 2, false);
        else E2M1_ROWS(1024, 1, false);
    } else if (units <= 2048) {
        if (many) E2M1_ROWS(512, 4, false);
        else E2M1_ROWS(1024, 2, false);
    } else {
        E2M1_ROWS(1024, 2, true);
    }
#undef E2M1_ROWS
    return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, bool bf16, int8_t* q, float* scale, int64_t rows, int64_t k,
                                hipStream_t stream) {
    return bf16 ? dispatch<uint16_t, kPlain>(x, nullptr, nullptr, 0.f, nullptr, q, scale, rows, k, stream)
                : dispatch<float, kPlain>(x, nullptr, nullptr, 0.f, nullptr, q, scale, rows, k, stream);
}

hipError_t launch_rmsnorm_int8_quantize(const void* x, const void* residual, const void* weight, bool bf16, float eps,
                                        void* residual_out, int8_t* q, float* scale, int64_t rows, int64_t k,
                                        hipStream_t stream) {
    if (residual != nullptr)
        return bf16 ? dispatch<uint16_t, kNormRes>(x, residual, weight, eps, residual_out, q, scale, rows, k, stream)
                    : dispatch<float, kNormRes>(x, residual, weight, eps, residual_out, q, scale, rows, k, stream);
    return bf16 ? dispatch<uint16_t, kNorm>(x, nullptr, weight, eps, nullptr, q, scale, rows, k, stream)
                : dispatch<float, kNorm>(x, nullptr, weight, eps, nullptr, q, scale, rows, k, stream);
}

hipError_t launch_silu_mul_int8_quantize(const void* gate_up, bool bf16, int8_t* q, float* scale, int64_t rows,
                                         int64_t inter, hipStream_t stream) {
    return bf16 ? dispatch<uint16_t, kAct>(gate_up, nullptr, nullptr, 0.f, nullptr, q, scale, rows, inter, stream)
                : dispatch<float, kAct>(gate_up, nullptr, nullptr, 0.f, nullptr, q, scale, rows, inter, stream);
}

}  // namespace e2m1
