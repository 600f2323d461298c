// k12_rows.cuh -- what the kernels that draw from rows of logits share: whole
// weights, the order of a row's tokens, block sums.
//
// A row's tokens are ordered by falling logit, equal ones by index.  Token i weighs
//   w_i = round(2^44 e^((x_i - max) / T)),
// a whole number, so that sums of weights are exact, the same in any order, and
// fit 64 bits (V <= 2^19): what is kept and drawn does not depend on how the
// row was shared out.  What a row keeps is then a first part of that order
// (min-p, top-k and top-p each cut its end), and a draw is the token where the
// running sum of weights passes u times the sum of those kept.
//
// 2^44 e^(-d / T) is computed in pairs of fp32 numbers: p = d log2(e) / T to 2^-47
// of itself, 2^(frac p) as a product of two table entries (7 bits each) and
// 1 + z + z^2 / 2 + z^3 / 6 with |z| < 2^-15, in 62-bit fixed point.  It is off
// by well under a unit below 2^42 and by 2^-44 of itself above.
#pragma once

#include "sdv_device.cuh"
#include "sdv_layer.h"
#include "sdv_plan.h"

namespace sdv {
namespace rows {

constexpr int kOneBits = 44;                 // the largest weight is 2^44
constexpr float kFallMost = 45.5f;           // a fall (in halvings) from which on a weight is 0

// 2^(i / 128) and 2^(i / 2^14) for i = -64 .. 64, in units of 2^-62.
constexpr double exp_series(double x) {
    double term = 1.0, sum = 1.0;
    for (int i = 1; i < 24; ++i) {
        term *= x / i;
        sum += term;
    }
    return sum;
}
struct Tables {
    uint64_t coarse[129], fine[129];
};
constexpr Tables make_tables() {
    Tables t{};
    for (int i = 0; i < 129; ++i) {
        const double ln2 = 0.693147180559945309417;
        t.coarse[i] = static_cast<uint64_t>(exp_series((i - 64) / 128.0 * ln2) * 4611686018427387904.0);
        t.fine[i] = static_cast<uint64_t>(exp_series((i - 64) / 16384.0 * ln2) * 4611686018427387904.0);
    }
    return t;
}
__device__ constexpr Tables kTables = make_tables();

// What turns a row's logits into weights.
struct Scale {
    float top;               // the row's largest logit
    float hi, lo;            // 2 log2(e) / T
};

__device__ __forceinline__ Scale scale_of(float top, float T) {
    Scale s;
    const double c = 2.8853900817779268147 / static_cast<double>(T);
    s.top = top;
    s.hi = static_cast<float>(c);
    s.lo = static_cast<float>(c - static_cast<double>(s.hi));
    return s;
}

// How far x lies below the largest, in halvings of the weight, as an fp32
// number; `low` is what it lacks.
__device__ __forceinline__ float fall_of(const Scale& s, float x, float& low) {
    // the halves' difference does not overflow; what its rounding loses is exact
    const float a = 0.5f * s.top, b = -0.5f * x;
    const float d = a + b, bb = d - a;
    const float e = (a - (d - bb)) + (b - bb);
    const float p = __fmul_rn(d, s.hi);
    low = __fmaf_rn(d, s.hi, -p) + __fmaf_rn(d, s.lo, __fmul_rn(e, s.hi));
    return p;
}

// The whole weight of a logit that is at most the largest.
__device__ __forceinline__ uint64_t weight_of(const Scale& s, float x, const Tables& t) {
    if (x == s.top) return uint64_t(1) << kOneBits;
    float low;
    const float p = fall_of(s, x, low);
    if (!(p < kFallMost)) return 0;
    const float k = rintf(p), f = k - p;                         // exact; 2^-p = 2^-k 2^f
    const int i = __float2int_rn(f * 128.0f);
    const float g = __fmaf_rn(static_cast<float>(i), -0x1p-7f, f);
    const int j = __float2int_rn(g * 16384.0f);
    const float h = __fmaf_rn(static_cast<float>(j), -0x1p-14f, g);
    const float z = h - low, zl = (h - z) - low;                 // |z| < 2^-14.9
    const float y = __fmul_rn(z, 0.693147182f);                  // z ln 2, and what that lacks
    const float yl = __fmaf_rn(z, 0.693147182f, -y) + __fmaf_rn(z, -1.90465421e-9f, __fmul_rn(zl, 0.693147182f));
    const float more = yl + __fmul_rn(__fmul_rn(y, y), __fmaf_rn(y, 0.166666667f, 0.5f));
    const int64_t one = int64_t(1) << 62;
    const uint64_t q = static_cast<uint64_t>(one + __float2ll_rn(y * 0x1p62f) + __float2ll_rn(more * 0x1p62f));
    const uint64_t ab = __umul64hi(t.coarse[i + 64], t.fine[j + 64]) << 2;
    const uint64_t w = __umul64hi(ab, q) << 2;                   // 2^f in units of 2^-62
    const int shift = 62 - kOneBits + static_cast<int>(k);       // 18 .. 63
    return ((w >> (shift - 1)) + 1) >> 1;
}

// Logits in order: a larger one has a larger key, and both zeros the same.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }
constexpr uint32_t kKeyLow = 0x007fffffu;    // -infinity
constexpr uint32_t kKeyHigh = 0xff800000u;   // +infinity; keys outside the two are not numbers

}  // namespace rows
}  // namespace sdv
