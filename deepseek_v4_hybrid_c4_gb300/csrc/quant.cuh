// The quantised latent row: 512 e4m3 codes and four e8m0 scales, one for each 128 dims (csa_quant_write).  A page
// holds its rows' codes one behind the other, then their scales.
#pragma once
#include "common.cuh"

namespace csa {

constexpr int Q_CODES = D, Q_SCALES = D / 128;
constexpr int Q_ROW_BYTES = Q_CODES + Q_SCALES;

// Codes of slot `slot` of page `page`, and its four scales.
CSA_DEV uint8_t* q_codes(const uint8_t* base, int64_t page_stride, int page, int slot) {
    return const_cast<uint8_t*>(base) + (int64_t)page * page_stride + (int64_t)slot * Q_CODES;
}
CSA_DEV uint8_t* q_scales(const uint8_t* base, int64_t page_stride, int rpp, int page, int slot) {
    return const_cast<uint8_t*>(base) + (int64_t)page * page_stride + (int64_t)rpp * Q_CODES + (int64_t)slot * Q_SCALES;
}

// What e4m3x4_bits() are to be multiplied by for a scale s, in both halves: 2^(s - 127 + 120), or NaN.  Above 2^127
// (s > 134) that is no bf16: the rest is q_factor_rest().
CSA_DEV uint32_t q_factor(uint32_t s) {
    const uint32_t h = s == 255u ? 0x7FC0u : min(s + 120u, 254u) << 7;
    return h * 0x10001u;
}
CSA_DEV uint32_t q_factor_rest(uint32_t s) { return (s > 134u && s < 255u ? (s - 7u) << 7 : 0x3F80u) * 0x10001u; }

CSA_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four e4m3 codes with their bits at their places in a bf16: sign, four bits of exponent, three of fraction.  As a
// bf16 that is the code's value times 2^-120, subnormals among them (both formats count those from their least
// exponent), so that one multiplication by a power of two is exact.  The codes 0x7F and 0xFF, which csa_quant_write does not
// make, become +-480 and no NaN here, where rows are read back: looking for them would be a third of the work on top.
// (cvt.rn.f16x2.e4m3x2, by which attention converts, has NaN for them.)
CSA_DEV uint2 e4m3x4_bits(uint32_t w) {
    const uint32_t lo = __byte_perm(w, 0, 0x1404), hi = __byte_perm(w, 0, 0x3424);
    return make_uint2((lo & 0x80008000u) | ((lo >> 4) & 0x07F007F0u), (hi & 0x80008000u) | ((hi >> 4) & 0x07F007F0u));
}

// 0x7F80 at the places of those bf16 whose codes are 0x7F or 0xFF.
CSA_DEV uint2 e4m3x4_nan(uint32_t w) {
    const uint32_t n = ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    const uint32_t lo = __byte_perm(n, 0, 0x1404), hi = __byte_perm(n, 0, 0x3424);
    return make_uint2(lo - (lo >> 8), hi - (hi >> 8));
}

// 16 codes as 16 bf16 (two uint4).
CSA_DEV void q_values(const uint4& c, uint32_t f, uint4& a, uint4& b) {
    const uint2 x = e4m3x4_bits(c.x), y = e4m3x4_bits(c.y), z = e4m3x4_bits(c.z), w = e4m3x4_bits(c.w);
    a = make_uint4(mul_bf16x2(x.x, f), mul_bf16x2(x.y, f), mul_bf16x2(y.x, f), mul_bf16x2(y.y, f));
    b = make_uint4(mul_bf16x2(z.x, f), mul_bf16x2(z.y, f), mul_bf16x2(w.x, f), mul_bf16x2(w.y, f));
}
CSA_DEV void q_times(uint4& a, uint32_t f) {
    a = make_uint4(mul_bf16x2(a.x, f), mul_bf16x2(a.y, f), mul_bf16x2(a.z, f), mul_bf16x2(a.w, f));
}

// The largest of a row's four scales (bytes of w) that is a number; 127 where none is.
CSA_DEV uint32_t q_top(uint32_t w) {
    const uint32_t nan = ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u;  // of bytes of 255
    if (nan) w &= ~((nan >> 7) * 255u);
    const uint32_t m = __vmaxu2(w & 0x00FF00FFu, (w >> 8) & 0x00FF00FFu);
    return nan == 0x80808080u ? 127u : max(m & 255u, m >> 16);
}
CSA_DEV uint32_t q_power(uint32_t s) { return s ? s << 23 : 0x00400000u; }  // 2^(s - 127), fp32
// 2^Q_UP times scale s over 2^(top - 127), in fp16: a value is at most 480 * 2^Q_UP, and the least ratio that there is
// 2^-24, so that a block is lost only where its scale is 2^32 and more below (2^25 without Q_UP).  A block 2^22 and more below
// loses bits of its smallest codes: at most 2^-32 of the larger unit.
constexpr int Q_UP = 7;
CSA_DEV uint32_t q_ratio(uint32_t s, uint32_t top) {
    const int d = (int)(top - s) - Q_UP;
    return s == 255u ? 0x7E00u : d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u;
}

static __device__ __noinline__ uint2 q_ratios_any(uint32_t w, uint32_t top) {
    return make_uint2(q_ratio(w & 255u, top) | q_ratio((w >> 8) & 255u, top) << 16,
                      q_ratio((w >> 16) & 255u, top) | q_ratio(w >> 24, top) << 16);
}
// Those of a row's four scales, all numbers (0 where the row is not there).  As a rule no block is 2^15 below: the upper
// bytes are (15 + Q_UP - d) << 2, all four at once.
CSA_DEV uint2 q_ratios(uint32_t w, uint32_t top, bool there) {
    const uint32_t d = top * 0x01010101u - w, h = ((15 + Q_UP) * 0x01010101u - d) << 2;
    uint2 r = make_uint2(__byte_perm(h, 0, 0x1404), __byte_perm(h, 0, 0x3424));
    if (!there) r = make_uint2(0, 0);
    else if ((d + 0x01010101u) & 0xF0F0F0F0u) r = q_ratios_any(w, top);
    return r;
}
CSA_DEV float q_log(uint32_t power) { return (float)(int)(power >> 23) - 127.f; }  // s - 127 of q_power(s)

// 16 codes as 16 fp16 (two uint4), times r (an fp16's bits).
CSA_DEV void e4m3x4_f16(uint32_t c, __half2 r, uint32_t& a, uint32_t& b) {
    uint32_t t, u;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(t), "=r"(u)
        : "r"(c));
    const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&t), r), y = __hmul2(*reinterpret_cast<__half2*>(&u), r);
    a = *reinterpret_cast<const uint32_t*>(&x);
    b = *reinterpret_cast<const uint32_t*>(&y);
}
CSA_DEV void q_halves(const uint4& c, uint32_t bits, uint4& a, uint4& b) {
    const __half2 r = __half2half2(__ushort_as_half((unsigned short)bits));
    e4m3x4_f16(c.x, r, a.x, a.y);
    e4m3x4_f16(c.y, r, a.z, a.w);
    e4m3x4_f16(c.z, r, b.x, b.y);
    e4m3x4_f16(c.w, r, b.z, b.w);
}

// Values of 2^128 and more, which are infinities as bf16: 2^Q_UP times the least of them over a row's largest scale, in
// fp16 (infinity where the row has none).
CSA_DEV uint32_t q_limit(uint32_t top) { return top >= 247u ? (270u + Q_UP - top) << 10 : 0x7C00u; }

// The last sequence that starts at or before row `row` (a warp; B + 1 offsets that do not fall): 32 of those left
// are looked at a time.
CSA_DEV int warp_seq_of(const int64_t* offsets, int B, int64_t row, int lane) {
    int l = 0, n = B;
    while (n > 1) {
        const int step = (n + 31) / 32, at = l + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, lane * step < n && __ldg(offsets + at) <= row);
        const int k = m ? 31 - __clz((int)m) : 0;
        l += k * step;
        n = min(step, n - k * step);
    }
    return l;
}

}  // namespace csa
