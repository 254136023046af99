// Keys that order tokens by their logits, and weights exp(logit - the largest)
// in fixed point; shared by sampling and beam selection.  (No FP64 here: a few
// instructions of it in every thread cost more than a pass over the logits.)
#pragma once
#include "dev_serve.cuh"

namespace mk {

constexpr uint64_t KEY_NONE = ~0ull;
// Keys rise in sampling order: the larger logit first, then the lower index.
DEV uint32_t ordered_bits(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
DEV unsigned long long sample_key(float x, int i) {
    return ((unsigned long long)(~ordered_bits(x)) << 32) | (uint32_t)i;
}

// 2^31 2^(-i/32)
static __constant__ uint32_t c_table[32] = {
    2147483648u, 2101467502u, 2056437387u, 2012372174u, 1969251188u, 1927054196u, 1885761398u, 1845353420u,
    1805811301u, 1767116489u, 1729250827u, 1692196547u, 1655936265u, 1620452965u, 1585730000u, 1551751076u,
    1518500250u, 1485961921u, 1454120821u, 1422962010u, 1392470869u, 1362633090u, 1333434672u, 1304861917u,
    1276901417u, 1249540052u, 1222764986u, 1196563654u, 1170923762u, 1145833280u, 1121280436u, 1097253708u};

// 2^44 2^-d for d >= 0 in 32.32 fixed point, below 2^31.
DEV unsigned long long octave_weight(long long d, const uint32_t *table) {
    const uint32_t f = (uint32_t)d;
    // 2^-f = table x exp(-a), a = (f mod 1/32) ln 2 < 0.0217: terms to a^4 / 24 leave 4e-11
    const uint32_t a = __umulhi(f & 0x07ffffffu, 2977044472u);  // ln 2 in 0.32
    uint32_t q = 715827883u - __umulhi(a, 178956971u);         // 1/6 - a/24
    q = 0x80000000u - __umulhi(a, q);                          // 1/2 - a q
    q = 0xffffffffu - __umulhi(a, q);                          // 1 - a q
    const uint32_t e = 0x80000000u - (__umulhi(a, q) >> 1);    // 1 - a q, in 1.31
    const unsigned long long prod = (unsigned long long)table[f >> 27] * e;  // 2.62
    return prod >> min(18 + (int)(d >> 32), 63);
}

// 2^44 2^-d in 64-bit fixed point, accurate to 2^-30 of itself or to 2^-44.
struct Weigher {
    float top, ch, cl;  // the row's maximum; log2(e) / temperature as a pair of fp32
    const uint32_t *table;
    DEV float octaves(float x) const { return (top - x) * ch; }  // d in fp32: monotone in x
    // d in 32.32 fixed point for d < most, else most + 1 (most: below 127); not for the largest itself, which may be infinite
    DEV long long distance(float x, float most) const {
        const float dh = top - x;
        const float bp = dh - top;
        const float dl = (top - (dh - bp)) + (-x - bp);  // dh + dl = top - x exactly
        const float t = fminf(dh * ch, most + 1.f);      // (NaN too)
        const float te = t < most ? fmaf(dh, ch, -t) + fmaf(dh, cl, dl * ch) : 0.f;
        const int n = __float2int_rz(t);
        // t - n is exact, te below 2^-16
        return max(0ll, ((long long)n << 32) + (long long)__float2uint_rz((t - (float)n) * 4294967296.f) +
                                         (long long)__float2int_rn(te * 4294967296.f));
    }
    // 2^44 2^-d, without branches, so that several weights overlap; from d = 46 on it is 0
    DEV unsigned long long operator()(float x) const {
        const unsigned long long r = octave_weight(distance(x, 46.f), table);
        return x == top ? 1ull << 44 : r;  // (the largest may be infinite)
    }
};

DEV unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}

}  // namespace mk
