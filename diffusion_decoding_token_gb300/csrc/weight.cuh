// weight.cuh -- softmax weights in 64-bit fixed point (sm_103a; the arithmetic
// also compiles for the host, where the tests compare it with 64-bit floats).
//
// A sampled token is the first whose running sum of weights exceeds u times
// their total, so a running sum has to be on the right side of a border that
// may lie anywhere.  With 32-bit sums (error ~1e-7 of the total) a flat row of
// 10^5 tokens, each 10^-5 of the total, misses in about one row of a hundred.
// Here a weight is an integer in units of 2^-44 with a relative error below
// 2^-37: sums of integers are exact and do not depend on their order, and a
// border is missed in less than one of 10^6 such rows.
//
//   w = 2^-y,  y = (m - z) log2(e) / T >= 0 in two floats (an exact difference
//   times a two-float constant), k = round(256 y), w = 2^-(k div 256) *
//   tab[k mod 256] * 2^-r with |r| <= 2^-9, and 2^-r = 1 - g + g^2/2 - g^3/6,
//   g = r ln 2, in integers of 2^-39 (the next term is below 2^-42).
// About 35 instructions, so it is used where few weights decide (the tokens
// that a filter keeps) or where a 32-bit pass can not tell.
#pragma once

#include <stdint.h>

#ifndef __CUDACC__
#include <math.h>
#include <string.h>
#define DLM_HD inline
#else
#define DLM_HD __device__ __forceinline__
#endif

namespace dlm {

constexpr int kWeightBits = 44;       // one unit is 2^-44 of the largest weight
constexpr float kUnit = 5.684341886080802e-14f;  // 2^-44
constexpr float kWeightCut = 46.0f;   // below 2^-46 a weight rounds to 0

// round(2^44 * 2^(-j/256))
#ifdef __CUDACC__
static __device__ const uint64_t kPow2Neg[256] = {
#else
static const uint64_t kPow2Neg[256] = {
#endif
    0x100000000000ull, 0x0ff4ecb59512ull, 0x0fe9e115c7b9ull, 0x0fdedd1b496bull,
    0x0fd3e0c0cf48ull, 0x0fc8ec01121eull, 0x0fbdfed6ce5full, 0x0fb3193cc422ull,
    0x0fa83b2db723ull, 0x0f9d64a46eb9ull, 0x0f92959bb5ddull, 0x0f87ce0e5b21ull,
    0x0f7d0df730adull, 0x0f7255510c43ull, 0x0f67a416c734ull, 0x0f5cfa433e65ull,
    0x0f5257d15248ull, 0x0f47bcbbe6dcull, 0x0f3d28fde3a6ull, 0x0f329c9233b7ull,
    0x0f281773c5a0ull, 0x0f1d999d8b77ull, 0x0f13230a7ad1ull, 0x0f08b3b58cbfull,
    0x0efe4b99bdceull, 0x0ef3eab20e03ull, 0x0ee990f980daull, 0x0edf3e6b1d42ull,
    0x0ed4f301ed99ull, 0x0ecaaeb8ffb0ull, 0x0ec0718b64c2ull, 0x0eb63b743173ull,
    0x0eac0c6e7dd2ull, 0x0ea1e4756551ull, 0x0e97c38406c5ull, 0x0e8da9958465ull,
    0x0e8396a503c5ull, 0x0e798aadadd6ull, 0x0e6f85aaaee2ull, 0x0e658797368bull,
    0x0e5b906e77c8ull, 0x0e51a02ba8e2ull, 0x0e47b6ca0374ull, 0x0e3dd444c465ull,
    0x0e33f8972be9ull, 0x0e2a23bc7d7eull, 0x0e2055afffe8ull, 0x0e168e6cfd33ull,
    0x0e0ccdeec2a9ull, 0x0e031430a0daull, 0x0df9612deb8full, 0x0defb4e1f9d1ull,
    0x0de60f4825e1ull, 0x0ddc705bcd38ull, 0x0dd2d8185083ull, 0x0dc9467913a5ull,
    0x0dbfbb797dafull, 0x0db63714f8e3ull, 0x0dacb946f2adull, 0x0da3420adba5ull,
    0x0d99d15c278bull, 0x0d9067364d45ull, 0x0d870394c6dbull, 0x0d7da6731179ull,
    0x0d744fccad6aull, 0x0d6aff9d1e14ull, 0x0d61b5dfe9faull, 0x0d5872909ab7ull,
    0x0d4f35aabcffull, 0x0d45ff29e097ull, 0x0d3ccf09985aull, 0x0d33a5457a30ull,
    0x0d2a81d91f13ull, 0x0d2164c02305ull, 0x0d184df62517ull, 0x0d0f3d76c75cull,
    0x0d06333daef3ull, 0x0cfd2f4683f9ull, 0x0cf4318cf192ull, 0x0ceb3a0ca5dcull,
    0x0ce248c151f8ull, 0x0cd95da6a9ffull, 0x0cd078b86504ull, 0x0cc799f23d11ull,
    0x0cbec14fef27ull, 0x0cb5eecd3b38ull, 0x0cad2265e429ull, 0x0ca45c15afccull,
    0x0c9b9bd866e3ull, 0x0c92e1a9d518ull, 0x0c8a2d85c900ull, 0x0c817f681416ull,
    0x0c78d74c8abcull, 0x0c70352f0433ull, 0x0c67990b5aa2ull, 0x0c5f02dd6b0cull,
    0x0c5672a11550ull, 0x0c4de8523c2cull, 0x0c4563ecc533ull, 0x0c3ce56c98d2ull,
    0x0c346ccda249ull, 0x0c2bfa0bcfaeull, 0x0c238d2311e4ull, 0x0c1b260f5ca1ull,
    0x0c12c4cca667ull, 0x0c0a6956e883ull, 0x0c0213aa1f0dull, 0x0bf9c3c248e2ull,
    0x0bf1799b67a7ull, 0x0be935317fc3ull, 0x0be0f6809861ull, 0x0bd8bd84bb68ull,
    0x0bd08a39f581ull, 0x0bc85c9c560eull, 0x0bc034a7ef2full, 0x0bb81258d5b7ull,
    0x0baff5ab2134ull, 0x0ba7de9aebe6ull, 0x0b9fcd2452c1ull, 0x0b97c1437568ull,
    0x0b8fbaf47630ull, 0x0b87ba337a17ull, 0x0b7fbefca8caull, 0x0b77c94c2c9dull,
    0x0b6fd91e328dull, 0x0b67ee6eea3bull, 0x0b60093a85edull, 0x0b58297d3a8cull,
    0x0b504f333f9eull, 0x0b487a58cf4bull, 0x0b40aaea2655ull, 0x0b38e0e3841aull,
    0x0b311c412a91ull, 0x0b295cff5e48ull, 0x0b21a31a6662ull, 0x0b19ee8e8c95ull,
    0x0b123f581d2bull, 0x0b0a957366fbull, 0x0b02f0dcbb6eull, 0x0afb51906e76ull,
    0x0af3b78ad691ull, 0x0aec22c84cc6ull, 0x0ae493452ca3ull, 0x0add08fdd43dull,
    0x0ad583eea42aull, 0x0ace0413ff84ull, 0x0ac6896a4be4ull, 0x0abf13edf162ull,
    0x0ab7a39b5a94ull, 0x0ab0386ef488ull, 0x0aa8d2652ec9ull, 0x0aa1717a7b57ull,
    0x0a9a15ab4ea8ull, 0x0a92bef41fa7ull, 0x0a8b6d5167b3ull, 0x0a8420bfa299ull,
    0x0a7cd93b4e96ull, 0x0a7596c0ec56ull, 0x0a6e594cfeefull, 0x0a6720dc0be1ull,
    0x0a5fed6a9b15ull, 0x0a58bef536dcull, 0x0a5195786beaull, 0x0a4a70f0c957ull,
    0x0a43515ae09eull, 0x0a3c36b34599ull, 0x0a3520f68e80ull, 0x0a2e102153e9ull,
    0x0a27043030c5ull, 0x0a1ffd1fc25dull, 0x0a18faeca854ull, 0x0a11fd9384a3ull,
    0x0a0b0510fb97ull, 0x0a041161b3d0ull, 0x09fd22825640ull, 0x09f6386f8e29ull,
    0x09ef5326091aull, 0x09e872a276f1ull, 0x09e196e189d4ull, 0x09dabfdff636ull,
    0x09d3ed9a72d0ull, 0x09cd200db8a0ull, 0x09c6573682ecull, 0x09bf93118f3bull,
    0x09b8d39b9d55ull, 0x09b218d16f44ull, 0x09ab62afc950ull, 0x09a4b13371fdull,
    0x099e0459320bull, 0x09975c1dd475ull, 0x0990b87e266cull, 0x098a1976f759ull,
    0x09837f0518dcull, 0x097ce9255ec4ull, 0x097657d49f18ull, 0x096fcb0fb20bull,
    0x096942d37202ull, 0x0962bf1cbb8eull, 0x095c3fe86d6dull, 0x0955c5336888ull,
    0x094f4efa8fefull, 0x0948dd3ac8deull, 0x09426ff0fab2ull, 0x093c071a0ef0ull,
    0x0935a2b2f13eull, 0x092f42b88f67ull, 0x0928e727d953ull, 0x09228ffdc10aull,
    0x091c3d373ab1ull, 0x0915eed13c89ull, 0x090fa4c8beeeull, 0x09095f1abc54ull,
    0x09031dc43146ull, 0x08fce0c21c67ull, 0x08f6a8117e6dull, 0x08f073af5a20ull,
    0x08ea4398b45dull, 0x08e417ca940eull, 0x08ddf042022eull, 0x08d7ccfc09c5ull,
    0x08d1adf5b7e6ull, 0x08cb932c1bafull, 0x08c57c9c4647ull, 0x08bf6a434adeull,
    0x08b95c1e3ea9ull, 0x08b3522a38e2ull, 0x08ad4c6452c7ull, 0x08a74ac9a799ull,
    0x08a14d575497ull, 0x089b540a7902ull, 0x08955ee03619ull, 0x088f6dd5af15ull,
    0x088980e8092eull, 0x088398146b92ull, 0x087db357ff6aull, 0x0877d2afefd5ull,
    0x0871f61969e9ull, 0x086c1d919cafull, 0x08664915b924ull, 0x086078a2f236ull,
    0x085aac367cc5ull, 0x0854e3cd8f9dull, 0x084f1f65637aull, 0x08495efb3304ull,
    0x0843a28c3aceull, 0x083dea15b954ull, 0x08383594eefbull, 0x083285071e10ull,
    0x082cd8698ac3ull, 0x08272fb97b2aull, 0x08218af43740ull, 0x081bea1708deull,
    0x08164d1f3bc0ull, 0x0810b40a1d81ull, 0x080b1ed4fd9aull, 0x08058d7d2d5eull,
};

// The row's constants: the maximum and log2(e) / T as a sum of two floats, and
// where the table lies (a kernel's copy in shared memory, or the constant one).
struct WeightScale {
    float m, c_hi, c_lo;
    const uint64_t* tab;
};

// log2(e) / T to 2^-47: a float quotient and its remainder's.
DLM_HD WeightScale weight_scale(float m, float temperature) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2(e)
    WeightScale s;
    s.m = m;
    s.c_hi = kHi / temperature;
    s.c_lo = (fmaf(-s.c_hi, temperature, kHi) + kLo) / temperature;
    s.tab = kPow2Neg;
    return s;
}

// y = (m - z) log2(e) / T as hi + lo; lo is meaningless when hi is infinite.
DLM_HD float weight_exponent(float z, const WeightScale& s, float& lo) {
    const float d = s.m - z;
    const float y = d * s.c_hi;
    // what the difference lost: m - z = d + err exactly
    const float b = d - s.m;
    const float err = (s.m - (d - b)) + (-z - b);
    float e = fmaf(d, s.c_hi, -y);
    e = fmaf(d, s.c_lo, e);
    lo = fmaf(err, s.c_hi, e);
    return y;
}

// 2^-(y + e) in units of 2^-44, y >= 0 and e small against 2^-9.
DLM_HD uint64_t weight44_of(float y, float e, const uint64_t* table = kPow2Neg) {
    if (!(y < kWeightCut)) return 0;
    constexpr float kMagic = 49152.0f;  // 1.5 * 2^15: its last place is 2^-8
    const float t = y + kMagic;
#ifdef __CUDA_ARCH__
    const int k = __float_as_int(t) - __float_as_int(kMagic);
    const float r = y - (t - kMagic);  // exact
    const int R = __float2int_rn(r * 549755813888.0f) + __float2int_rn(e * 549755813888.0f);
#else
    const int k = (int)((t - kMagic) * 256.0f);
    const float r = y - (t - kMagic);
    const int R = (int)rintf(r * 549755813888.0f) + (int)rintf(e * 549755813888.0f);
#endif
    const int g = (int)(((int64_t)R * 2977044472ll) >> 32);  // ln 2 in 2^-32
    const int g2 = (int)(((int64_t)g * g) >> 40);
    const float gf = (float)g;
    const int g3 = (int)(gf * gf * gf * 5.5145374e-25f);  // 2^-78 / 6
    const int q = g2 - g - g3;
    const uint64_t tab = table[k & 255];
    const uint64_t w = tab + (uint64_t)(((int64_t)(tab >> 13) * q) >> 26);
    const int n = k >> 8;
    return (w + ((1ull << n) >> 1)) >> n;
}

// exp((z - m) / T) in units of 2^-44, z <= m; 0 for z = -inf and for NaN.
DLM_HD uint64_t weight44(float z, const WeightScale& s) {
    float e;
    const float y = weight_exponent(z, s, e);
    return weight44_of(y, e, s.tab);
}

// ln x to 2^-36 for any normal x > 0: with x = m 2^e and m in [1, 2), the float
// logarithm y of m is off by what m 2^-y is off 1 by, 2^-y from the integer
// weights.  (Of x itself that product would have no digits left: from x = 2^25 on
// the logarithm was off by more than 2^-18, from 2^46 on by 1.5.  64-bit arithmetic
// has a 64th of the 32-bit rate here: a double logarithm by every thread of a CTA
// took 7 us.)
DLM_HD double log_exact(float x) {
#ifdef __CUDA_ARCH__
    const uint32_t b = __float_as_uint(x);
    const float m = __uint_as_float((b & 0x7fffffu) | 0x3f800000u), y = fmaxf(0.f, __log2f(m));
#else
    uint32_t b;
    memcpy(&b, &x, 4);
    const uint32_t mb = (b & 0x7fffffu) | 0x3f800000u;
    float m;
    memcpy(&m, &mb, 4);
    const float y = fmaxf(0.f, log2f(m));
#endif
    const double d = (double)m * ((double)weight44_of(y, 0.f) * (double)kUnit) - 1.0;
    return ((double)((int)(b >> 23) - 127) + (double)y) * 0.6931471805599453 + (d - 0.5 * d * d);
}

// floor(f * s) for a float f in [0, 1): f = mantissa * 2^-shift exactly.
// `inexact` says whether anything was cut off.
DLM_HD uint64_t scale_floor(uint64_t s, float f, bool& inexact) {
#ifdef __CUDA_ARCH__
    const uint32_t b = __float_as_uint(f);
#else
    uint32_t b;
    memcpy(&b, &f, 4);
#endif
    const int ex = (int)(b >> 23) & 255;
    const uint64_t mant = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int shift = 150 - (ex ? ex : 1);  // 24 .. 149
#ifdef __CUDA_ARCH__
    const uint64_t hi = __umul64hi(s, mant);
#else
    const uint64_t hi = (uint64_t)(((unsigned __int128)s * mant) >> 64);
#endif
    const uint64_t lo = s * mant;
    if (shift >= 128) {
        inexact = (hi | lo) != 0;
        return 0;
    }
    if (shift >= 64) {
        const int r = shift - 64;
        inexact = lo != 0 || (r ? (hi & ((1ull << r) - 1)) : 0) != 0;
        return hi >> r;
    }
    inexact = (lo & ((1ull << shift) - 1)) != 0;
    return (hi << (64 - shift)) | (lo >> shift);
}

// The smallest integer that is at least f * s.
DLM_HD uint64_t scale_ceil(uint64_t s, float f) {
    bool inexact;
    const uint64_t x = scale_floor(s, f, inexact);
    return x + (inexact ? 1 : 0);
}

}  // namespace dlm
