// kda_wide.cuh -- sums and comparisons of about 48 bits from fp32 instructions, for choices that hang on the last
// digits: a value is a pair of fp32, hi + lo.  fp64 would be the plain way, but an fp64 instruction holds a
// warp's scheduler for 16 cycles on sm_103, and its results come late.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

// A running sum: hi as fp32 adds it, lo what the additions lost.
struct Sum2 {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float s = hi + v, b = s - hi;
        lo += (hi - (s - b)) + (v - b);
        hi = s;
    }
};

// A pair whose lo is at most half a step of hi, so that pairs compare part by part.  A hi that is not finite
// has lo = 0.
struct Wide {
    float hi = 0.f, lo = 0.f;
};
__device__ __forceinline__ Wide wide(float hi, float lo) {  // |hi| >= |lo|
    const float s = hi + lo;
    return Wide{s, fabsf(s) < INFINITY ? lo - (s - hi) : 0.f};
}
__device__ __forceinline__ Wide wide(const Sum2& s) { return wide(s.hi, s.lo); }
__device__ __forceinline__ Wide add(Wide a, Wide b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    return wide(s, (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo));
}
__device__ __forceinline__ Wide minus(Wide a) { return Wide{-a.hi, -a.lo}; }
__device__ __forceinline__ Wide times(Wide a, Wide b) {
    const float p = a.hi * b.hi;
    return wide(p, fmaf(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
__device__ __forceinline__ bool above(Wide a, Wide b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Wide from(unsigned lanes, Wide v, int src) {
    return Wide{__shfl_sync(lanes, v.hi, src), __shfl_sync(lanes, v.lo, src)};
}

__device__ __forceinline__ Wide over(Wide a, Wide b) {  // one Newton step from the fp32 quotient
    const float q = a.hi / b.hi;
    const Wide left = add(a, minus(times(Wide{q, 0.f}, b)));
    return wide(q, (left.hi + left.lo) / b.hi);
}

// e^m for m <= 0 to about 45 bits.  With n the integer next to m log2(e) and r = m - n ln 2 (|r| < 0.35), e^r is its
// Taylor series: 14 terms leave 0.35^15 / 15! < 2^-62; the last terms are too small for their pairs' second halves to
// count.  Below -80 the fp32 value: it is less than any digit kept of a sum with a 1 in it.
__device__ __forceinline__ Wide exp_wide(Wide m) {
    if (!(m.hi >= -80.f)) return Wide{expf(m.hi), 0.f};
    const float n = rintf(m.hi * 1.4426950408889634f);
    // ln 2 in three parts (Cody and Waite's reduction): the first two of 13 and 17 bits, so that their products with n
    // (at most 116) are exact
    constexpr float kLn2Top = 0.693115234375f, kLn2Mid = 0x1.0bfbp-15f;
    constexpr float kLn2Rest = (float)(0.69314718055994530942 - (double)kLn2Top - (double)kLn2Mid);
    Wide r = wide(fmaf(-n, kLn2Top, m.hi), 0.f);
    r = add(r, Wide{-n * kLn2Mid, 0.f});
    r = add(r, Wide{m.lo, 0.f});
    r = add(r, Wide{-n * kLn2Rest, 0.f});
    float tail = 1.1470745597729725e-11f;  // 1 / 14!
    tail = fmaf(tail, r.hi, 1.6059043836821613e-10f);
    tail = fmaf(tail, r.hi, 2.08767569878681e-09f);
    tail = fmaf(tail, r.hi, 2.505210838544172e-08f);
    tail = fmaf(tail, r.hi, 2.755731922398589e-07f);  // 1 / 10!
    Wide p = wide(2.755731922398589e-06f, tail * r.hi);
    constexpr double kInv[9] = {1.0, 1.0, 0.5, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320};
#pragma unroll
    for (int i = 8; i >= 0; --i) {
        const float c = (float)kInv[i];
        p = add(Wide{c, (float)(kInv[i] - (double)c)}, times(p, r));
    }
    const float scale = __int_as_float(((int)n + 127) << 23);  // n in [-116, 0]
    return Wide{p.hi * scale, p.lo * scale};
}

// To the 53 bits of an fp64: what differs by less is equal.
__device__ __forceinline__ Wide to_53_bits(Wide a) {
    const uint32_t e = __float_as_uint(a.hi) >> 23 & 0xffu;
    if (e < 30u || e == 255u) return a;
    const float c = 1.5f * __uint_as_float((e - 29u) << 23);  // fp32 of this size steps by 2^-52 of hi's power of two
    return Wide{a.hi, __fsub_rn(__fadd_rn(a.lo, c), c)};
}

// 1 / (1 + e^-x) to about 45 bits.
__device__ __forceinline__ Wide sigmoid_wide(Wide x) {
    if (isnan(x.hi)) return x;
    const bool positive = x.hi > 0.f;
    const Wide e = exp_wide(positive ? minus(x) : x);  // at most 1
    return over(positive ? Wide{1.f, 0.f} : e, add(Wide{1.f, 0.f}, e));
}

}  // namespace kda
