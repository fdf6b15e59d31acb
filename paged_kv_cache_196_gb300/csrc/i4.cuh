// The 4-bit cache format (KV_I4): how a tile is laid out, how values become
// codes and codes values.
//
// 16 consecutive dimensions of one (token, kv head) are a group: sixteen
// integer codes c in -7..7 and one e4m3 scale s, standing for c * s * g with g
// the pool's power-of-two scale of K or V.  s is the e4m3 nearest to
// max|x| / (7 g) (at most 448), c the integer nearest to x / (s g), both ties to
// even; a group whose s rounds to 0 holds zeros, a group with a NaN is NaN.
// c * s has at most 7 significant bits and lies between 2^-9 and 3136: exact in
// fp16 and bf16.
//
// A (block, kv head) tile of K or of V is 16 x D / 2 bytes of codes followed by
// 16 x D / 16 scale bytes (9 D bytes; 1152 for D = 128).  A K tile is followed by its V
// tile, so that one copy of 18 D bytes brings both.  A code is stored as u = c + 8 in
// four bits.
//   K  token t's row is D / 2 bytes in order of dimensions, dimension d in the
//      four bits d % 8 of the row's 32-bit word d / 8; its scale of group j is
//      byte t * D / 16 + j of the scales.  A lane of the score product loads a
//      quarter row, 16 consecutive bytes.
//   V  is contracted over tokens, so the two tokens of a pair (2p, 2p + 1) share
//      words: word (p, quad) holds dimensions 4 quad .. 4 quad + 3 of token 2p in
//      its low half and of token 2p + 1 in its high half, so that a masked word
//      is already the pair of operands the tensor core wants.  A token owns whole
//      16-bit halves and whole scale bytes: tokens of one pair may be written at the
//      same time.  Pair p's D / 4 words lie at word p D / 4, in an order that lets
//      the eight lanes (of four pairs) that load together hit all banks: quad q at
//      position q ^ v_swizzle(p).  Scales: byte p * D / 8 + 2 j + (t & 1).
//   A scale byte is the e4m3 code; NaN is 0xff, so that the byte shifted left by 7
//   is an fp16 NaN and otherwise the fp16 value s / 256 (see scale_pair).
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace pkv {
namespace i4 {

// Larger of two, NaN if either is.
KV_DEVICE float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The e4m3 nearest to x >= 0 (at most 448) as its byte; 0xff for NaN.
KV_DEVICE uint32_t e4m3_of(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return x != x ? 0xffu : r;
}

// Two e4m3 bytes (low byte first) as a pair of fp16 values, exact.
KV_DEVICE __half2 e4m3x2_to_half2(uint32_t b) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(b));
    return *reinterpret_cast<__half2 *>(&r);
}

KV_DEVICE float e4m3_to_float(uint32_t b) { return __low2float(e4m3x2_to_half2(b)); }

// Where pair p keeps its quad q: q ^ v_swizzle<D>(p).
template <int D>
KV_DEVICE constexpr int v_swizzle(int p) {
    return D == 128 ? 8 * (p & 3) : 8 * ((p >> 1) & 1);
}

// x / d from an approximate reciprocal r of d: a first quotient q = x r, its residual
// x - q d, and the correction q + (x - q d) r, Newton's step for the quotient in the form
// that a fused multiply-add allows (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", IBM J. Res. Dev. 34, 1990).
// Error: with r = (1 + e) / d, |e| <= 2^-22, q is x / d (1 + e') with |e'| <= |e| + 2^-24;
// the residual is exact (both terms are multiples of q's last place times d's, and their
// difference is small) and the correction leaves x / d (1 - e e'), so the result is the
// rounding of a number within 2^-43 of the quotient, relatively.
KV_DEVICE float divide(float x, float d, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
}

KV_DEVICE float reciprocal(float x) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The scale byte of a group with largest magnitude m.  A border b between two e4m3
// values has 5 significant bits, 7 b at most 8: m = 7 b comes out as b exactly, and an m
// one last place away is at least 4 / 7 of b's last place from b after the division
// (ulp(7 b) is 4 or 8 times ulp(b)), so it does not round to b.
KV_DEVICE uint32_t scale_byte(float m) {
    m = m > 1e30f ? 1e30f : m;  // an infinity would leave NaN; NaN stays
    return e4m3_of(divide(m, 7.f, 1.f / 7.f));
}

// Eight values of one group half -> their eight 4-bit codes, value i in bits
// 4i .. 4i + 3, given the group's scale s (a value of e4m3).
//
// c = rint(x / s) must be decided as exact arithmetic decides it: values of 16
// bits are often exactly between two codes.  A border (k + 1/2) s has at most 8
// significant bits: x on it gives k + 1/2 exactly.  An x one last place away is at
// least 8 / 15 of the quotient's last place from it after the division (s's mantissa is
// at most 15 / 8; a border that is a power of two has s a power of two, an exact
// division), so it does not round to it.  Clamping x to +-7.25 s
// first (exact) keeps infinities and |c| > 7 out.  rint and the bias are one addition
// of 1.5 * 2^23 + 8.
KV_DEVICE uint32_t codes8(const float (&x)[8], float s) {
    const float lim = 7.25f * s;
    const float r = s > 0.f ? reciprocal(s) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float q = divide(fminf(fmaxf(x[i], -lim), lim), s, r);
        // low bits of the sum's word: rint(q) + 8, in 1..15; the rest is the same in
        // each and subtracted once
        w = w * 16u + __float_as_uint(__fadd_rn(q, 12582920.f));
    }
    return w - 0x4B400000u * 0x11111111u;
}

// Two scale bytes (low byte first) as the fp16 pair s / 256.  e4m3's exponent and
// mantissa are the low bits of fp16's with a bias 8 smaller, so it is a shift, exact
// for every e4m3 (subnormals become fp16 subnormals); the byte 0xff becomes a NaN.
KV_DEVICE __half2 scale_pair(uint32_t two) {
    const uint32_t h = __byte_perm(two, 0u, 0x1404) >> 1;
    return *reinterpret_cast<const __half2 *>(&h);
}

// Four code pairs of one word as fp16 pairs times their scales (c s / 256): out[n]
// = (low half's four bits n, high half's four bits n).
//
// Four bits at the bottom of the mantissa of 1024, or above four zero bits in that of
// 64, give 1024 + u or 64 + u with one logical operation, and one fused multiply-add
// takes it to (u - 8) s: the constants -1032 s and -72 s are exact (129 and 9 times
// the four significant bits of s fit 11), the product is not rounded before the sum,
// and the result has 7 bits.
struct Scale {
    __half2 s, m72, m1032;
};

KV_DEVICE Scale make_scale(__half2 s) {
    Scale r;
    r.s = s;
    r.m72 = __hmul2(s, __float2half2_rn(-72.f));
    r.m1032 = __hmul2(s, __float2half2_rn(-1032.f));
    return r;
}

// (w & mask) | bits as one instruction.
KV_DEVICE uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}

KV_DEVICE uint32_t fma2(uint32_t x, __half2 s, __half2 m) {
    const __half2 v = __hfma2(*reinterpret_cast<const __half2 *>(&x), s, m);
    return *reinterpret_cast<const uint32_t *>(&v);
}

KV_DEVICE void values8(uint32_t w, const Scale &k, uint32_t (&out)[4]) {
    const uint32_t b = w >> 8;
    out[0] = fma2(and_or(w, 0x000F000Fu, 0x64006400u), k.s, k.m1032);
    out[1] = fma2(and_or(w, 0x00F000F0u, 0x54005400u), k.s, k.m72);
    out[2] = fma2(and_or(b, 0x000F000Fu, 0x64006400u), k.s, k.m1032);
    out[3] = fma2(and_or(b, 0x00F000F0u, 0x54005400u), k.s, k.m72);
}

// What values8 leaves out: the callers multiply their sums by it.
constexpr float kScaleUnit = 256.f;

}  // namespace i4
}  // namespace pkv
