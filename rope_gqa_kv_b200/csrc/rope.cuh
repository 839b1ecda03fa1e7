// rope.cuh -- what the kernels that normalise and rotate head vectors share: the
// frequency table, the rotation of one vector held by a group of lanes, and the
// programmatic-dependent launch.
#pragma once

#include <cmath>

#include "common.cuh"

namespace gqa {

// Rotation frequencies theta_i of the D/2 pairs (float64) and the factor the
// rotated vectors are multiplied by (1 except for YaRN).
struct RopeTable {
    double theta[64];
    float mscale;
};

template <int D>
struct RopeShape {
    static constexpr int kHalf = D / 2;
    static constexpr int kChunks = kHalf / 8;               // active lanes per vector
    static constexpr int kTPV = kChunks <= 4 ? 4 : 8;       // lanes per vector (pow2)
    static constexpr int kVecPerWarp = 32 / kTPV;
};

// Sum over the TPV-lane group (aligned, power of two) of this lane's value.
template <int TPV>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = TPV / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Two fp32 lanes at once (one issue slot each): d = a * b, d = a * b + c.
__device__ __forceinline__ void mul2(float &d0, float &d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float &d0, float &d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// cos / sin (times the YaRN factor) of the 8 rotation pairs 8j .. 8j+7 that
// lane j of a vector group owns, read from a row of D/2 angles in shared memory;
// zero on lanes that own no pair.
template <int D>
__device__ __forceinline__ void lane_angles(const float *cs_row, const float *sn_row, int j,
                                            bool active, float (&c)[8], float (&sv)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float4 cv = make_float4(0.f, 0.f, 0.f, 0.f), sq = cv;
        if (active) {
            cv = *reinterpret_cast<const float4 *>(cs_row + 8 * j + 4 * h);
            sq = *reinterpret_cast<const float4 *>(sn_row + 8 * j + 4 * h);
        }
        c[4 * h] = cv.x; c[4 * h + 1] = cv.y; c[4 * h + 2] = cv.z; c[4 * h + 3] = cv.w;
        sv[4 * h] = sq.x; sv[4 * h + 1] = sq.y; sv[4 * h + 2] = sq.z; sv[4 * h + 3] = sq.w;
    }
}

// RMSNorm (if qk_norm) and rotation of the lane's 16 coordinates.
template <int D>
__device__ __forceinline__ void rotate_vector(const uint4 a_in, const uint4 b_in, uint4 &a_out,
                                              uint4 &b_out, const float (&c)[8],
                                              const float (&sv)[8], bool active, bool qk_norm,
                                              float eps) {
    using S = RopeShape<D>;
    float xa[8], xb[8];
    const uint32_t wa[4] = {a_in.x, a_in.y, a_in.z, a_in.w};
    const uint32_t wb[4] = {b_in.x, b_in.y, b_in.z, b_in.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        xa[2 * e] = bf16lo(wa[e]);
        xa[2 * e + 1] = bf16hi(wa[e]);
        xb[2 * e] = bf16lo(wb[e]);
        xb[2 * e + 1] = bf16hi(wb[e]);
    }
    if (qk_norm) {
        // sum of squares and the scaling on coordinate pairs (packed f32x2)
        float s0 = 0.f, s1 = 0.f;
        if (active) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                fma2(s0, s1, xa[e], xa[e + 1], xa[e], xa[e + 1], s0, s1);
                fma2(s0, s1, xb[e], xb[e + 1], xb[e], xb[e + 1], s0, s1);
            }
        }
        const float ss = group_sum<S::kTPV>(s0 + s1);
        const float inv = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            mul2(xa[e], xa[e + 1], xa[e], xa[e + 1], inv, inv);
            mul2(xb[e], xb[e + 1], xb[e], xb[e + 1], inv, inv);
        }
    }
    // rotation of pairs (8j + 2e, 8j + 2e + 1) two at a time:
    //   ya = a c - b s,  yb = a s + b c
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float c0 = c[2 * e], c1 = c[2 * e + 1], s0 = sv[2 * e], s1 = sv[2 * e + 1];
        const float a0 = xa[2 * e], a1 = xa[2 * e + 1], b0 = xb[2 * e], b1 = xb[2 * e + 1];
        float ya0, ya1, yb0, yb1;
        mul2(ya0, ya1, b0, b1, -s0, -s1);
        fma2(ya0, ya1, a0, a1, c0, c1, ya0, ya1);
        mul2(yb0, yb1, b0, b1, c0, c1);
        fma2(yb0, yb1, a0, a1, s0, s1, yb0, yb1);
        oa[e] = pack_bf16x2(ya0, ya1);
        ob[e] = pack_bf16x2(yb0, yb1);
    }
    a_out = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    b_out = make_uint4(ob[0], ob[1], ob[2], ob[3]);
}

// theta_i for the chosen variant, in float64 on the host (formulas in gqa.h).
inline RopeTable compute_table(int D, const gqa_rope_params &p) {
    RopeTable t;
    const int half = D / 2;
    const double base = (double)p.rope_base, s = (double)p.factor;
    const double two_pi = 6.283185307179586476925286766559;
    double eff_base = base;
    if (p.scaling == GQA_ROPE_NTK) eff_base = base * std::pow(s, (double)D / (double)(D - 2));
    for (int i = 0; i < 64; ++i) t.theta[i] = 0.0;
    for (int i = 0; i < half; ++i) {
        const double th = std::pow(eff_base, -2.0 * (double)i / (double)D);
        double out = th;
        if (p.scaling == GQA_ROPE_LINEAR) {
            out = th / s;
        } else if (p.scaling == GQA_ROPE_YARN) {
            const double r = (double)p.original_max_pos * th / two_pi;
            double gmix = (r - (double)p.yarn_alpha) / ((double)p.yarn_beta - (double)p.yarn_alpha);
            gmix = gmix < 0.0 ? 0.0 : (gmix > 1.0 ? 1.0 : gmix);
            out = (1.0 - gmix) * th / s + gmix * th;
        }
        t.theta[i] = out;
    }
    t.mscale = p.scaling == GQA_ROPE_YARN ? (float)(0.1 * std::log(s) + 1.0) : 1.0f;
    return t;
}

// The same, computed again only when D or the parameters change: the 32 to 64 powers
// take about as long as a launch.
inline const RopeTable &make_table(int D, const gqa_rope_params &p) {
    struct Last {
        int D = 0;
        gqa_rope_params p = {};
        RopeTable t = {};
    };
    static thread_local Last last;
    const gqa_rope_params &q = last.p;
    if (last.D != D || q.rope_base != p.rope_base || q.scaling != p.scaling ||
        q.factor != p.factor || q.original_max_pos != p.original_max_pos ||
        q.yarn_alpha != p.yarn_alpha || q.yarn_beta != p.yarn_beta) {
        last.t = compute_table(D, p);
        last.D = D;
        last.p = p;
    }
    return last.t;
}

// A launch as a programmatic dependent of the preceding kernel on the stream: its
// launch overlaps that kernel's last CTAs (the kernel waits for it on entry).
template <typename K, typename... Args>
cudaError_t launch_pdl(K kern, dim3 grid, unsigned block, cudaStream_t s, Args... args) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

inline bool params_ok(const gqa_rope_params &p) {
    if (!(p.eps >= 0.f && p.rope_base > 1.f)) return false;
    switch (p.scaling) {
        case GQA_ROPE_PLAIN: return true;
        case GQA_ROPE_LINEAR:
        case GQA_ROPE_NTK: return p.factor >= 1.f;
        case GQA_ROPE_YARN:
            return p.factor >= 1.f && p.original_max_pos >= 1 && p.yarn_alpha >= 0.f &&
                   p.yarn_beta > p.yarn_alpha;
        default: return false;
    }
}

}  // namespace gqa
