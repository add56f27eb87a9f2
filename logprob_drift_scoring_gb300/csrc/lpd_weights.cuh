// Softmax weights as whole numbers: exp(scale (x - top)) in steps of 2^-45.
//
// A filter's border (the smallest prefix whose mass reaches top_p) and a draw
// (the first token whose running mass passes u W) compare sums that may lie
// arbitrarily near each other, so the sums of a row are integers: any order of
// addition gives the same bits, and one row's answer does not depend on how its
// columns were spread over threads.  A weight is formed to 2^-29.5 of itself
// (weight_rough) and for the row's heaviest tokens to 2^-41 (weight_precise):
// the errors of many small weights average out, those of a few large ones would
// not.  (A plain exponential in float32 is off by 2^-22 with the rounding of its
// argument: it moves the border of a nucleus by a token in one row of a thousand.)  What a
// weight has below a step is cut off: V light tokens take at most V 2^-45 of the top's weight
// from a sum, 2^-27.8 for 151936 of them.  (Rounded to the nearest step they are off by half of
// it, and float32 nuclei take 5 to 7 % longer; more bits have no room, 393216 weights of the
// top's size being 2^63.6.)
//
// x scale log2(e) is cut in units of 1/256 octave, x c = J + a with whole J and
// |a| <= 1/2; 2^(J / 256) comes from a table and shifts, 2^(a / 256) - 1 from
// three terms of its series (the fourth is below 2^-41).  The product x c is
// formed exactly with a multiply-add, so nothing is lost to the size of x.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#ifndef __CUDACC__
#define __host__
#define __device__
#define __forceinline__ inline
#endif

namespace lpd {

constexpr int kWeightOne = 45;          // weights are multiples of 2^-45 of the top's (about)
constexpr int kUnits = 256;             // steps an octave
constexpr float kMagic = 12582912.f;    // 1.5 * 2^23: adding it rounds to a whole number
constexpr uint32_t kMagicBits = 0x4b400000u;

struct WeightEntry {
    uint32_t whole;  // 2^(i / 256) in units of 2^-30
    float part;      // the same as a float
};

// One row's exponent factor and origin.
struct WeightScale {
    double c;        // units for 1.0 of x
    float ch, cl;    // c in two floats
    int origin;      // whole units of the top
    float cut;       // x at or below this weigh nothing
    int wide;        // the top lies beyond 2^20 units: products by float lose whole units, doubles do not
};

__host__ __device__ __forceinline__ uint32_t bits_of(float x) {
#ifdef __CUDA_ARCH__
    return __float_as_uint(x);
#else
    uint32_t u;
    memcpy(&u, &x, 4);
    return u;
#endif
}
__host__ __device__ __forceinline__ float mul_rn(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fmul_rn(a, b);
#else
    return a * b;
#endif
}
__host__ __device__ __forceinline__ float add_rn(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fadd_rn(a, b);
#else
    return a + b;
#endif
}
__host__ __device__ __forceinline__ float fma_rn(float a, float b, float c) {
#ifdef __CUDA_ARCH__
    return __fmaf_rn(a, b, c);
#else
    return std::fmaf(a, b, c);
#endif
}

// scale: finite and > 0; top: the row's largest logit, finite.
__host__ __device__ __forceinline__ WeightScale weight_scale(float scale, float top) {
    WeightScale w;
    // (log2(e) 256 in two floats; c is what the two parts say)
    constexpr double kC = 1.4426950408889634073599 * kUnits;
    constexpr float kHi = static_cast<float>(kC), kLo = static_cast<float>(kC - static_cast<double>(kHi));
    w.ch = mul_rn(scale, kHi);
    w.cl = fma_rn(scale, kLo, fma_rn(scale, kHi, -w.ch));
    w.wide = !(fabsf(top * w.ch) < 1048576.f) || !(w.ch < 1e30f) || !(w.ch > 1e-30f);
    w.c = w.wide ? static_cast<double>(scale) * kC : static_cast<double>(w.ch) + static_cast<double>(w.cl);
    // (a wide row's origin is the top itself: weight_precise)
    w.origin = w.wide ? 0 : static_cast<int>(bits_of(add_rn(mul_rn(top, w.ch), kMagic)) - kMagicBits);
    w.cut = top - (kWeightOne + 2) * static_cast<float>(kUnits) / w.ch;
    return w;
}

constexpr double kLn2Unit = 0.69314718055994530942 / kUnits;

// For x > w.cut and x <= top, not wide.
__host__ __device__ __forceinline__ uint64_t weight_rough(float x, const WeightScale &w, const WeightEntry *table) {
    const float p = mul_rn(x, w.ch);
    const float q = fma_rn(x, w.cl, fma_rn(x, w.ch, -p));
    const float b = add_rn(p, kMagic);
    const float a = add_rn(add_rn(p, -add_rn(b, -kMagic)), q);
    const int j = static_cast<int>(bits_of(b) - kMagicBits) - w.origin;
    constexpr float k1 = static_cast<float>(kLn2Unit), k2 = static_cast<float>(kLn2Unit * kLn2Unit / 2),
                    k3 = static_cast<float>(kLn2Unit * kLn2Unit * kLn2Unit / 6);
    const float y = mul_rn(a, fma_rn(a, fma_rn(a, k3, k2), k1));
    const WeightEntry e = table[j & (kUnits - 1)];
    const uint32_t m = e.whole + (bits_of(fma_rn(e.part, y, kMagic)) - kMagicBits);
    const int s = -(j >> 8);  // octaves below the top's
    return (static_cast<uint64_t>(m) << (kWeightOne - 30)) >> (s & 63);
}

// 2^45 times a float below 2^18 in magnitude, rounded to a whole number.
__host__ __device__ __forceinline__ int64_t steps_of(float x) {
#ifdef __CUDA_ARCH__
    return __float2ll_rn(x * static_cast<float>(uint64_t{1} << kWeightOne));
#else
    return static_cast<int64_t>(std::nearbyint(static_cast<double>(x) * static_cast<double>(uint64_t{1} << kWeightOne)));
#endif
}

// For finite x <= top.  The argument and the terms of the series are carried in
// two floats, the table's entries in 2^-62: 2^-41 of the weight in all (and 2^-55 for each
// unit that x itself lies from 0).
__host__ __device__ __forceinline__ uint64_t weight_precise(float x, const WeightScale &w, float top, const uint64_t *table) {
    float h, q;  // the argument's fraction of a unit
    int j;
    if (w.wide) {
        const double u = (static_cast<double>(x) - static_cast<double>(top)) * w.c;
        if (!(u > -(kWeightOne + 2.0) * kUnits)) return 0;
        const double whole = rint(u);
        j = static_cast<int>(whole);
        h = static_cast<float>(u - whole);
        q = static_cast<float>(u - whole - static_cast<double>(h));
    } else {
        if (!(x > w.cut)) return 0;
        const float p = mul_rn(x, w.ch);
        const float b = add_rn(p, kMagic);
        j = static_cast<int>(bits_of(b) - kMagicBits) - w.origin;
        h = add_rn(p, -add_rn(b, -kMagic));
        q = fma_rn(x, w.cl, fma_rn(x, w.ch, -p));
    }
    const float a = add_rn(h, q), al = add_rn(q, -add_rn(a, -h));
    constexpr float k1 = static_cast<float>(kLn2Unit), k1l = static_cast<float>(kLn2Unit - static_cast<double>(k1)),
                    k2 = static_cast<float>(kLn2Unit * kLn2Unit / 2), k3 = static_cast<float>(kLn2Unit * kLn2Unit * kLn2Unit / 6),
                    k4 = static_cast<float>(kLn2Unit * kLn2Unit * kLn2Unit * kLn2Unit / 24);
    const float y = mul_rn(a, k1);
    const float yl = fma_rn(mul_rn(a, a), fma_rn(a, fma_rn(a, k4, k3), k2), fma_rn(al, k1, fma_rn(a, k1l, fma_rn(a, k1, -y))));
    const uint64_t t = table[j & (kUnits - 1)];  // 2^(i / 256) in units of 2^-62
    const float th = static_cast<float>(static_cast<uint32_t>(t >> 40)) * 2.384185791015625e-7f;  // its first 23 bits: 2^-22 each
    const float tl = static_cast<float>(static_cast<uint32_t>(t >> 8)) * 5.551115123125783e-17f;
    const float m = mul_rn(th, y);
    const float ml = fma_rn(tl, y, fma_rn(th, yl, fma_rn(th, y, -m)));
    const int s = -(j >> 8);
    const uint64_t v = ((t + (1u << (61 - kWeightOne))) >> (62 - kWeightOne)) + static_cast<uint64_t>(steps_of(m) + steps_of(ml));
    return v >> (s & 63);
}

}  // namespace lpd
