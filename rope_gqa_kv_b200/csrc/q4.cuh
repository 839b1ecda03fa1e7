// q4.cuh -- the 4-bit cache row: its layout and the quantiser.
//
// A row is the D values of one token of one KV head, in NG = D/32 groups; group g
// holds the rotation pairs 16 g .. 16 g + 15, i.e. coordinates i and i + D/2 of
// each (the two that RoPE mixes share a range, and so a scale).  Per group the row
// keeps a pair of bf16 numbers (s, m), and per value a code c in 0 .. 15 that
// stands for m + s c:
//     m = min x,   s = bf16((max x - m) / 15),   c = ceil((x - m) / s - 1/2).
// The values quantised are bf16, so m is exact; rounding s to 8 bits moves the
// largest value's quotient by at most 15 * 2^-8 = 0.06, so no code is clipped.  With
// the formula's codes |m + s c - x| <= s/2 for every value; q4_quantise lets a quotient
// less than 2^-19 of itself above n + 1/2 fall to n, which adds that share of the
// quotient times s, 15 * 2^-19 s at most.  A group with s below 2^-126 keeps
// s = 0 (all values m); one that holds a value that is not finite keeps m = NaN,
// s = 0: all its values read back as NaN.
//
// Codes (D/2 bytes): pair p = 16 g + 4 k + t has its byte -- coordinate p in the
// low four bits, p + D/2 in the high four -- at 4 * (NG * k + g) + t.  A row is
// thus four blocks of NG words, block k holding word k of every group: lane
// 4 r + k of a warp that loads block k of row r reads NG consecutive words, eight
// rows are one linear read, and each lane holds one word of every group, which is
// the shape of an mma.m16n8k16 operand (decode_q4.cu).
// Scales (4 NG bytes): word g = s in the low half, m in the high half.
#pragma once

#include "common.cuh"

namespace gqa {

template <int D>
struct Q4Shape {
    static constexpr int NG = D / 32;             // groups of a row
    static constexpr int kCodeBytes = D / 2;
};

// 2^-126 as fp32: smaller steps are not kept.
constexpr float kQ4MinStep = 1.17549435e-38f;

__device__ __forceinline__ uint32_t min_bf16x2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_bf16x2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// d = a * b + c on two fp32 lanes.
__device__ __forceinline__ void q4_fma2(float &d0, float &d1, float a0, float a1, float b,
                                        float c) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmov.b64 rc, {%5, %5};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}

// Quantises the 16 bf16 values a lane holds of one group: a = coordinates
// 8 j .. 8 j + 7, b = D/2 + the same; lanes j and j ^ 1 hold a group together and
// both must be converged here with every lane of the warp.  Returns this lane's
// two words of codes (pairs 8 j .. 8 j + 3 and 8 j + 4 .. 8 j + 7) and the group's
// (s, m) word.
//
// Halves are worked on so that max - m cannot overflow: t = (x - m) / 2 is one
// fused operation, exact whenever the difference fits 24 bits.  The quotient is
// t * (2/s) with 2/s made smaller by 2^-21 of itself: a quotient that is exactly
// n + 1/2 then lands below it by more than the rounding errors (2^-23) and rounds
// down to n, as the formula asks.  So does one that lies above n + 1/2 by less than
// that margin: x - m, of two bf16 values, can have more bits than fp32 (m = -s/2 and
// x = 2^-30 s have the quotient 1/2 + 2^-30, whose code would be 1).  Adding 1.5 * 2^23
// in the same fused operation leaves the rounded code in the low bits of the sum.
__device__ __forceinline__ void q4_quantise(const uint4 a, const uint4 b, uint32_t (&codes)[2],
                                            uint32_t &sm) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t lo = w[0], hi = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = min_bf16x2_nan(lo, w[i]);
        hi = max_bf16x2_nan(hi, w[i]);
    }
    lo = min_bf16x2_nan(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    hi = max_bf16x2_nan(hi, __shfl_xor_sync(0xffffffffu, hi, 1));
    lo = min_bf16x2_nan(lo, __byte_perm(lo, lo, 0x1032));
    hi = max_bf16x2_nan(hi, __byte_perm(hi, hi, 0x1032));
    const float mn = bf16hi(lo), mx = bf16hi(hi);
    const float half_range = fmaf(mx, 0.5f, -0.5f * mn);
    const bool finite = half_range < INFINITY;                  // false for NaN too
    const float step = bf16lo(pack_bf16x2(__fdiv_rn(half_range, 7.5f), 0.f));
    const bool live = finite && step >= kQ4MinStep;
    const float inv = live ? __fdiv_rn(2.0f, step) * (1.0f - 0x1p-21f) : 0.f;
    const uint32_t s_bits = live ? __float_as_uint(step) >> 16 : 0u;
    const uint32_t m_bits = finite ? (lo & 0xffff0000u) : 0x7fc00000u;
    sm = s_bits | m_bits;
    const uint32_t keep = live ? 0xffffffffu : 0u;
    const float mhalf = -0.5f * mn;
    uint32_t byte[8];                                           // low byte: one pair's codes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x0, x1, y0, y1;
        q4_fma2(x0, x1, bf16lo(w[i]), bf16hi(w[i]), 0.5f, mhalf);
        q4_fma2(y0, y1, bf16lo(w[4 + i]), bf16hi(w[4 + i]), 0.5f, mhalf);
        q4_fma2(x0, x1, x0, x1, inv, 12582912.0f);
        q4_fma2(y0, y1, y0, y1, inv, 12582912.0f);
        byte[2 * i] = __float_as_uint(x0) + (__float_as_uint(y0) << 4);
        byte[2 * i + 1] = __float_as_uint(x1) + (__float_as_uint(y1) << 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t p = __byte_perm(byte[4 * i], byte[4 * i + 1], 0x0040);
        const uint32_t q = __byte_perm(byte[4 * i + 2], byte[4 * i + 3], 0x0040);
        codes[i] = __byte_perm(p, q, 0x5410) & keep;
    }
}

}  // namespace gqa
