// norm_rope.cu -- per-head RMSNorm with learned gains, rotation by positions on up
// to four axes, and the write into a bf16 or a 4-bit cache, in one pass; and the
// backward of the bf16 form.
//
//   u = gain * x * (mean x^2 + eps)^(-1/2),   y = mscale * R(P) u,
//   pair i (coordinates i, i + D/2) turned by P_i theta_i, P_i the token's position
//   on pair i's axis (image and video tokens: time, height, width).
//
// Forward.  Bound by memory: q is read and written once, k and v read once, the
// cache rows written once.  A vector is held by 4 or 8 lanes, lane j with coordinates
// 8j .. 8j+7 and D/2 + 8j ..: both members of its 8 rotation pairs, and half of one
// group of the 4-bit row, so rotation needs no exchange, the norm one shuffle sum
// and the quantiser one shuffle per group.  A warp takes one token at a time (or, when
// there are few tokens, one slice of a token's vectors, so that a decode step still
// spreads over the SMs); it walks the token's query, key and value vectors
// kVecPerWarp at a time, a pass of one kind each.  What a lane needs of the next kRing
// passes, those of the warp's next tokens included, is on its way into the lane's own
// places of a shared-memory ring: the loads wait neither for the angles nor for the
// arithmetic, hold no registers, and each lane waits for its own alone.
#include "q4.cuh"
#include "rope.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 4;              // warps per CTA
// Measured on 8 x 2048 tokens of 24 / 8 heads, D = 128 (335 MB, 51 us at the copy rate):
// 62 us, 82 % of it; rings of 2, 4 and 8 passes 71, 65 and 64 us (longer ones leave less
// L1 for positions), 6 CTAs an SM 65 us.
constexpr int kResident = 5;           // CTAs per SM
constexpr int kRing = 3;               // passes on their way or waiting, per warp

struct AxisTable {
    uint8_t axis[64];
};

struct AppendArgs {
    const uint16_t *q, *k, *v;
    uint16_t *q_out;
    uint16_t *kc, *vc;                 // bf16 cache
    uint8_t *k_codes, *v_codes;        // 4-bit cache
    uint32_t *k_scales, *v_scales;
    const uint16_t *q_gain, *k_gain;
    const int32_t *pos0, *n_tok, *pos;
    int32_t *new_len, *status;
    int B, T, Hq, Hkv, Lmax, n_slices; // slices of a token's passes
    int qk_norm;
    float eps;
};

// The token's positions on the axes of the pairs that the lane works out: pairs lane and
// lane + 32.
template <int D>
struct Positions {
    static constexpr int N = (D / 2 + 31) / 32;
    int p[N];

    __device__ __forceinline__ void load(const int32_t *pos, int p_seq, int B, int T, int b, int t,
                                         const AxisTable &ax, int lane) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int i = lane + 32 * n;
            p[n] = p_seq;
            if (pos && i < D / 2) p[n] = pos[((size_t)ax.axis[i] * B + b) * T + t];
        }
    }
};

// cos / sin of the token's D/2 angles into the warp's rows: position times theta_i
// in float64, reduced to [-pi, pi] in float64, then fp32.
template <int D>
__device__ __forceinline__ void token_angles(float *cs, float *sn, const Positions<D> &pos,
                                             const RopeTable &tab, int lane) {
#pragma unroll
    for (int n = 0; n < Positions<D>::N; ++n) {
        const int i = lane + 32 * n;
        if (i >= D / 2) break;
        const double a = (double)pos.p[n] * tab.theta[i];
        const double two_pi = 6.283185307179586476925286766559;
        const double r = a - rint(a * (1.0 / two_pi)) * two_pi;
        float sf, cf;
        sincosf((float)r, &sf, &cf);
        cs[i] = cf * tab.mscale;
        sn[i] = sf * tab.mscale;
    }
}

// The CTA's gains as fp32 rows [q | k] in shared memory (ones where none is given).
template <int D>
__device__ __forceinline__ void load_gains(float (*gain)[D], const uint16_t *qg,
                                           const uint16_t *kg, int tid, int threads) {
    for (int i = tid; i < 2 * D; i += threads) {
        const uint16_t *src = i < D ? qg : kg;
        const int d = i < D ? i : i - D;
        gain[i / D][d] = src ? __uint_as_float((uint32_t)src[d] << 16) : 1.0f;
    }
}

// The rotation of the lane's 8 pairs (a, b) with the gains folded in:
//   ya = a (ga c) - b (gb s),   yb = a (ga s) + b (gb c).
struct Turn {
    float ac[8], nbs[8], as[8], bc[8];                     // nbs = -gb s
};

template <int D>
__device__ __forceinline__ void make_turn(Turn &t, const float *cs, const float *sn,
                                          const float *gain, int j, bool active) {
    float c[8], s[8];
    lane_angles<D>(cs, sn, j, active, c, s);
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        float4 ga = make_float4(0.f, 0.f, 0.f, 0.f), gb = ga;
        if (active) {
            ga = *reinterpret_cast<const float4 *>(gain + 8 * j + h);
            gb = *reinterpret_cast<const float4 *>(gain + D / 2 + 8 * j + h);
        }
        const float a[4] = {ga.x, ga.y, ga.z, ga.w}, b[4] = {gb.x, gb.y, gb.z, gb.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            t.ac[h + e] = a[e] * c[h + e];
            t.as[h + e] = a[e] * s[h + e];
            t.bc[h + e] = b[e] * c[h + e];
            t.nbs[h + e] = -(b[e] * s[h + e]);
        }
    }
}

// RMSNorm (if qk_norm) and rotation of the lane's 16 coordinates; with gains of one the
// bits of rotate_vector.  Lanes without a vector hold zeros.
template <int D>
__device__ __forceinline__ void turn_vector(uint4 &a, uint4 &b, const Turn &t, bool qk_norm,
                                            float eps) {
    using S = RopeShape<D>;
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
    float xa[8], xb[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        xa[2 * e] = bf16lo(wa[e]);
        xa[2 * e + 1] = bf16hi(wa[e]);
        xb[2 * e] = bf16lo(wb[e]);
        xb[2 * e + 1] = bf16hi(wb[e]);
    }
    if (qk_norm) {
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            fma2(s0, s1, xa[e], xa[e + 1], xa[e], xa[e + 1], s0, s1);
            fma2(s0, s1, xb[e], xb[e + 1], xb[e], xb[e + 1], s0, s1);
        }
        const float inv = rsqrtf(group_sum<S::kTPV>(s0 + s1) * (1.0f / D) + eps);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            mul2(xa[e], xa[e + 1], xa[e], xa[e + 1], inv, inv);
            mul2(xb[e], xb[e + 1], xb[e], xb[e + 1], inv, inv);
        }
    }
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        float ya0, ya1, yb0, yb1;
        mul2(ya0, ya1, xb[e], xb[e + 1], t.nbs[e], t.nbs[e + 1]);
        fma2(ya0, ya1, xa[e], xa[e + 1], t.ac[e], t.ac[e + 1], ya0, ya1);
        mul2(yb0, yb1, xb[e], xb[e + 1], t.bc[e], t.bc[e + 1]);
        fma2(yb0, yb1, xa[e], xa[e + 1], t.as[e], t.as[e + 1], yb0, yb1);
        oa[e / 2] = pack_bf16x2(ya0, ya1);
        ob[e / 2] = pack_bf16x2(yb0, yb1);
    }
    a = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    b = make_uint4(ob[0], ob[1], ob[2], ob[3]);
}

// A warp's way through its units -- unit, unit + stride, .. -- a unit being a slice of a
// token's passes: the slice, its token t of sequence b.  The steps are taken without a
// division.
struct Walk {
    int b, t, slice;
    int step_b, step_t, step_slice;

    __device__ __forceinline__ void start(unsigned unit, unsigned stride, int n_slices, int T) {
        const unsigned tok = unit / (unsigned)n_slices, step = stride / (unsigned)n_slices;
        slice = (int)(unit - tok * n_slices);
        step_slice = (int)(stride - step * n_slices);
        b = (int)(tok / (unsigned)T);
        step_b = (int)(step / (unsigned)T);
        t = (int)(tok - (unsigned)b * T);
        step_t = (int)(step - (unsigned)step_b * T);
    }
    __device__ __forceinline__ void step(int n_slices, int T) {
        b += step_b;
        t += step_t;
        slice += step_slice;
        if (slice >= n_slices) {
            slice -= n_slices;
            ++t;
        }
        if (t >= T) {
            t -= T;
            ++b;
        }
    }
};

// On to the first unit whose token is to be written; false behind the last.
__device__ __forceinline__ bool find_live(Walk &w, const AppendArgs &A, int &slot_row) {
    for (; w.b < A.B; w.step(A.n_slices, A.T)) {
        const int p0 = A.pos0 ? A.pos0[w.b] : 0;
        const int n = A.n_tok ? A.n_tok[w.b] : A.T;
        slot_row = p0 + w.t;
        if (p0 >= 0 && n >= 0 && n <= A.T && (long long)p0 + n <= A.Lmax && w.t < n) return true;
    }
    return false;
}

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32, kResident)
norm_rope_append_kernel(const AppendArgs A, const __grid_constant__ RopeTable tab,
                        const __grid_constant__ AxisTable ax) {
    using S = RopeShape<D>;
    using R = Q4Shape<D>;
    __shared__ __align__(16) uint4 ring[kWarps][kRing][2][32];
    __shared__ __align__(16) float cs[kWarps][S::kHalf];
    __shared__ __align__(16) float sn[kWarps][S::kHalf];
    __shared__ __align__(16) float gain[2][D];
    // A programmatic dependent of the kernel before it, which may have produced any
    // of its inputs: wait for that kernel to complete before reading.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = lane % S::kTPV;
    const int slot = lane / S::kTPV;
    const bool active = j < S::kChunks;
    // Passes of one kind each: query heads, then key heads, then value heads.
    const int nq = A.q ? A.Hq : 0;
    const int qp = (nq + S::kVecPerWarp - 1) / S::kVecPerWarp;
    const int kp = (A.Hkv + S::kVecPerWarp - 1) / S::kVecPerWarp;
    const int npass = qp + 2 * kp;

    Walk ahead;                        // of the loads
    ahead.start(blockIdx.x * kWarps + warp, gridDim.x * kWarps, A.n_slices, A.T);
    Walk at = ahead;                   // of the arithmetic
    const uint32_t mine = static_cast<uint32_t>(__cvta_generic_to_shared(&ring[warp][0][0][lane]));
    const int step_h = A.n_slices * S::kVecPerWarp;        // heads from pass to pass
    int row_ahead = 0;
    bool more = find_live(ahead, A, row_ahead);
    int ps_ahead = ahead.slice, end_ahead = 0;             // next pass, end of its kind
    int left_ahead = 0;                                    // heads of its kind from the lane's on
    const uint16_t *src = nullptr;
    // Starts the loads of the next pass, into a stage; always one commit group.
    auto load_next = [&](int stage) {
        if (more) {                                        // uniform across the warp
            if (ps_ahead >= end_ahead) {                   // the first pass of a kind
                const bool is_q = ps_ahead < qp, is_k = !is_q && ps_ahead < qp + kp;
                end_ahead = is_q ? qp : is_k ? qp + kp : npass;
                const int h = (ps_ahead - (is_q ? 0 : is_k ? qp : qp + kp)) * S::kVecPerWarp + slot;
                const int heads = is_q ? A.Hq : A.Hkv;
                const size_t tok = (size_t)ahead.b * A.T + ahead.t;
                src = (is_q ? A.q : is_k ? A.k : A.v) + (tok * heads + h) * D + 8 * j;
                left_ahead = active ? heads - h : 0;
            }
            if (left_ahead > 0) {
                copy16(mine + stage * 1024, src);
                copy16(mine + stage * 1024 + 512, src + S::kHalf);
            }
            src += (size_t)step_h * D;
            left_ahead -= step_h;
            ps_ahead += A.n_slices;
            if (ps_ahead >= npass) {
                ahead.step(A.n_slices, A.T);
                more = find_live(ahead, A, row_ahead);
                ps_ahead = ahead.slice;
                end_ahead = 0;
            }
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kRing - 1; ++i) load_next(i);

    // Lengths and errors of the sequences.
    for (int b = blockIdx.x * kWarps * 32 + threadIdx.x; b < A.B; b += gridDim.x * kWarps * 32) {
        const int p0 = A.pos0 ? A.pos0[b] : 0;
        const int n = A.n_tok ? A.n_tok[b] : A.T;
        const bool bad = p0 < 0 || n < 0 || n > A.T;
        const long long end = (long long)p0 + (n < 0 || n > A.T ? 0 : n);
        if (bad) report(A.status, GQA_DEV_BAD_LEN);
        else if (end > A.Lmax) report(A.status, GQA_DEV_CAPACITY);
        if (A.new_len) A.new_len[b] = (int)(end < 0x7fffffffLL ? end : 0x7fffffffLL);
    }
    load_gains<D>(gain, A.q_gain, A.k_gain, threadIdx.x, kWarps * 32);
    __syncthreads();                                       // only warp-level sync follows

    int stage = 0;
#pragma unroll 1
    for (int slot_row = 0; find_live(at, A, slot_row); at.step(A.n_slices, A.T)) {
        const int b = at.b;
        const size_t tok = (size_t)b * A.T + at.t;
        Positions<D> pos;
        pos.load(A.pos, slot_row, A.B, A.T, b, at.t, ax, lane);
        __syncwarp();                                      // the last unit's angles are read
        token_angles<D>(cs[warp], sn[warp], pos, tab, lane);
        __syncwarp();
        Turn turn;
        int end = 0, left = 0;                             // as of the loads
        bool is_q = false, is_k = false;
        uint16_t *dst = nullptr;                           // the lane's first chunk (not Q4's K, V)
        size_t row = 0;                                    // the cache row
#pragma unroll 1
        for (int ps = at.slice; ps < npass; ps += A.n_slices) {
            if (ps >= end) {                               // the first pass of a kind: uniform
                is_q = ps < qp;
                is_k = !is_q && ps < qp + kp;
                end = is_q ? qp : is_k ? qp + kp : npass;
                const int h = (ps - (is_q ? 0 : is_k ? qp : qp + kp)) * S::kVecPerWarp + slot;
                left = active ? (is_q ? A.Hq : A.Hkv) - h : 0;
                row = ((size_t)b * A.Hkv + h) * A.Lmax + slot_row;
                if (is_q) dst = A.q_out + (tok * A.Hq + h) * D + 8 * j;
                else if (!Q4) dst = (is_k ? A.kc : A.vc) + row * D + 8 * j;
                if (is_q || is_k) make_turn<D>(turn, cs[warp], sn[warp], gain[is_k], j, active);
            }
            copy_wait<kRing - 2>();
            uint4 a = make_uint4(0, 0, 0, 0), bb = a;
            const bool mem = left > 0;
            if (mem) {
                a = ring[warp][stage][0][lane];
                bb = ring[warp][stage][1][lane];
            }
            load_next(stage == 0 ? kRing - 1 : stage - 1); // the stage read before this one
            stage = stage == kRing - 1 ? 0 : stage + 1;
            if (is_q || is_k) turn_vector<D>(a, bb, turn, A.qk_norm != 0, A.eps);
            if (!Q4 || is_q) {
                if (mem) {
                    *reinterpret_cast<uint4 *>(dst) = a;
                    *reinterpret_cast<uint4 *>(dst + S::kHalf) = bb;
                }
                dst += (size_t)step_h * D * (is_q ? 1 : A.Lmax);
            } else {
                uint32_t codes[2], sm;
                q4_quantise(a, bb, codes, sm);
                if (mem) {
                    const int g = j >> 1, k0 = 2 * (j & 1);
                    uint32_t *cw = reinterpret_cast<uint32_t *>(is_k ? A.k_codes : A.v_codes) +
                                   row * (R::kCodeBytes / 4);
                    cw[R::NG * k0 + g] = codes[0];
                    cw[R::NG * (k0 + 1) + g] = codes[1];
                    if ((j & 1) == 0) (is_k ? A.k_scales : A.v_scales)[row * R::NG + g] = sm;
                }
                row += (size_t)step_h * A.Lmax;
            }
            left -= step_h;
        }
    }
    copy_wait<0>();
}

// ---------------------------------------------------------------------------
// backward of the bf16 form
// ---------------------------------------------------------------------------
// With r = (mean x^2 + eps)^(-1/2), dy the gradient of the rotated vector and
// w = mscale R(P)^T dy:
//   d gain = sum over tokens and heads of w x r,     z = gain w,
//   dx = r z - x r^3 mean(x z)          (without the norm: dx = w),
// and dv is the cache's gradient rows brought back to token order.
//
// Bound by memory: x, dy read once and dx written once.  The loads go through rings as
// in the forward.  A CTA takes either query passes or key and value passes, of tokens
// (or slices of them) in turn, so that a lane keeps one gain and the sums of one gain's
// gradient, for its 16 coordinates, in registers over all its units.  At the end a CTA
// adds its warps' sums and leaves one row in the workspace, and a second kernel adds the
// rows in a fixed order, so equal calls give equal bits.
//
// Measured on 8 x 2048 tokens of 24 / 8 heads, D = 128 (470 MB, 72 us at the copy rate):
// 82 to 90 us from GPU to GPU, 80 to 88 % of it; 4 CTAs an SM at fewer registers 97 us where
// this takes 82; 3 x 1001 tokens of 8 / 8 heads, D = 96 (5.6 us) 17 us, 3 of them the second
// kernel.
constexpr int kBwdWarps = 4;
constexpr int kBwdResident = 3;                            // CTAs per SM
constexpr int kBwdMaxCtas = 148 * kBwdResident;
constexpr int kBwdRing = 4;                                // passes on their way or waiting
constexpr uint32_t kNoVector = 0x3f803f80u;                // x where there is none: two bf16 ones

struct BackwardArgs {
    const uint16_t *q, *k, *dq_out, *dkc, *dvc;
    uint16_t *dq, *dk, *dv;
    const uint16_t *q_gain, *k_gain;
    const int32_t *pos0, *pos;
    float *partial;                    // [CTAs][D], NULL: no gain gradients wanted
    int32_t *status;
    int B, T, Hq, Hkv, Lmax;
    int n_q;                           // CTAs of the query passes; the rest: keys and values
    int slices[2];                     // slices of a token's passes: query, key and value
    int qk_norm;
    float eps;
};

// One vector: dx of the lane's 16 coordinates in place of dy (ya, yb), and its share of
// d gain added to dg.  Lanes without a vector hold dy = 0 and x = 1 (kNoVector): of zeros r
// would be infinite with eps = 0, and their share of d gain NaN.
template <int D>
__device__ __forceinline__ void backward_vector(const uint4 xa, const uint4 xb, uint4 &ya,
                                                uint4 &yb, const float (&c)[8],
                                                const float (&s)[8], bool qk_norm, float eps,
                                                const float (&gain)[16], float (&dg)[16]) {
    using S = RopeShape<D>;
    const uint32_t xw[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
    const uint32_t yw[8] = {ya.x, ya.y, ya.z, ya.w, yb.x, yb.y, yb.z, yb.w};
    float w[16];                       // [0..7] first-half chunk, [8..15] second-half chunk
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a0 = bf16lo(yw[e]), a1 = bf16hi(yw[e]);
        const float b0 = bf16lo(yw[4 + e]), b1 = bf16hi(yw[4 + e]);
        const float c0 = c[2 * e], c1 = c[2 * e + 1], s0 = s[2 * e], s1 = s[2 * e + 1];
        mul2(w[2 * e], w[2 * e + 1], b0, b1, s0, s1);
        fma2(w[2 * e], w[2 * e + 1], a0, a1, c0, c1, w[2 * e], w[2 * e + 1]);
        mul2(w[8 + 2 * e], w[9 + 2 * e], a0, a1, -s0, -s1);
        fma2(w[8 + 2 * e], w[9 + 2 * e], b0, b1, c0, c1, w[8 + 2 * e], w[9 + 2 * e]);
    }
    if (qk_norm) {                     // uniform
        float ss0 = 0.f, ss1 = 0.f, xz0 = 0.f, xz1 = 0.f;
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float x0 = bf16lo(xw[e / 2]), x1 = bf16hi(xw[e / 2]);
            float z0, z1;
            fma2(ss0, ss1, x0, x1, x0, x1, ss0, ss1);
            mul2(z0, z1, w[e], w[e + 1], gain[e], gain[e + 1]);
            fma2(xz0, xz1, x0, x1, z0, z1, xz0, xz1);
        }
        const float ss = group_sum<S::kTPV>(ss0 + ss1);
        const float xz = group_sum<S::kTPV>(xz0 + xz1);
        const float r = rsqrtf(ss * (1.0f / D) + eps);
        const float k = -r * (xz * r * (1.0f / D));        // r^3 alone could overflow
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            float t0, t1, z0, z1;
            mul2(t0, t1, bf16lo(xw[e / 2]), bf16hi(xw[e / 2]), r, r);
            fma2(dg[e], dg[e + 1], w[e], w[e + 1], t0, t1, dg[e], dg[e + 1]);
            mul2(z0, z1, w[e], w[e + 1], gain[e], gain[e + 1]);
            mul2(t0, t1, t0, t1, k, k);
            fma2(w[e], w[e + 1], z0, z1, r, r, t0, t1);
        }
    }
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = pack_bf16x2(w[2 * e], w[2 * e + 1]);
    ya = make_uint4(o[0], o[1], o[2], o[3]);
    yb = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D>
struct BackwardShared {
    uint4 ring[kBwdWarps][kBwdRing][4][32];                // dy, dy, x, x
    float cs[kBwdWarps][D / 2], sn[kBwdWarps][D / 2];
    float sums[kBwdWarps][D];
};

// The warp's units: query passes (QUERIES) or key passes, then value passes.
template <int D, bool QUERIES>
__device__ __forceinline__ void backward_units(const BackwardArgs &A, const RopeTable &tab,
                                               const AxisTable &ax, BackwardShared<D> &sh) {
    using S = RopeShape<D>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = lane % S::kTPV, slot = lane / S::kTPV;
    const bool active = j < S::kChunks;
    const int heads = QUERIES ? A.Hq : A.Hkv;
    const int per_kind = (heads + S::kVecPerWarp - 1) / S::kVecPerWarp;
    const int npass = QUERIES ? per_kind : 2 * per_kind;
    const int n_slices = A.slices[QUERIES ? 0 : 1];
    const int cta = QUERIES ? (int)blockIdx.x : (int)blockIdx.x - A.n_q;
    const unsigned stride = (QUERIES ? A.n_q : gridDim.x - A.n_q) * kBwdWarps;
    const bool norm = A.qk_norm != 0;
    const uint32_t fill = active ? kNoVector : 0u;         // lanes beyond D/16 add nothing to a norm

    float gain[16], dg[16];
    {
        const uint16_t *g = QUERIES ? A.q_gain : A.k_gain;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int d = (e < 8 ? 0 : S::kHalf) + 8 * j + (e & 7);
            gain[e] = !active ? 0.f : g ? __uint_as_float((uint32_t)g[d] << 16) : 1.0f;
            dg[e] = 0.f;
        }
    }

    // On to the first unit in range; false behind the last.
    auto find = [&](Walk &w, int &slot_row) {
        for (; w.b < A.B; w.step(n_slices, A.T)) {
            const int p0 = A.pos0 ? A.pos0[w.b] : 0;
            slot_row = p0 + w.t;
            if (p0 >= 0 && (long long)p0 + A.T <= A.Lmax) return true;
        }
        return false;
    };
    const int step_h = n_slices * S::kVecPerWarp;          // heads from pass to pass
    const size_t x_step = (size_t)step_h * D, y_step = QUERIES ? x_step : x_step * A.Lmax;

    // The loads, kBwdRing - 1 passes ahead of the arithmetic.
    Walk ahead;
    ahead.start(cta * kBwdWarps + warp, stride, n_slices, A.T);
    Walk next = ahead;                 // of the arithmetic
    int slot_row = 0, kend = 0, kleft = 0;
    bool more = find(ahead, slot_row);
    int kps = ahead.slice;
    const uint16_t *xs = nullptr, *ys = nullptr;
    const uint32_t mine =
        static_cast<uint32_t>(__cvta_generic_to_shared(&sh.ring[warp][0][0][lane]));
    auto load_next = [&](int stage) {
        if (more) {                                        // uniform across the warp
            const bool value = !QUERIES && kps >= per_kind;
            if (kps >= kend) {                             // the first pass of a kind
                kend = value ? npass : per_kind;
                const int h = (value ? kps - per_kind : kps) * S::kVecPerWarp + slot;
                const size_t in = (((size_t)ahead.b * A.T + ahead.t) * heads + h) * D + 8 * j;
                const size_t row = (((size_t)ahead.b * A.Hkv + h) * A.Lmax + slot_row) * D + 8 * j;
                xs = (QUERIES ? A.q : A.k) + in;
                ys = QUERIES ? A.dq_out + in : (value ? A.dvc : A.dkc) + row;
                kleft = active ? heads - h : 0;
            }
            if (kleft > 0) {
                const uint32_t dst = mine + stage * 2048;
                copy16(dst, ys);
                copy16(dst + 512, ys + S::kHalf);
                if (norm && !value) {
                    copy16(dst + 1024, xs);
                    copy16(dst + 1536, xs + S::kHalf);
                }
            }
            xs += x_step;
            ys += y_step;
            kleft -= step_h;
            kps += n_slices;
            if (kps >= npass) {
                ahead.step(n_slices, A.T);
                more = find(ahead, slot_row);
                kps = ahead.slice;
                kend = 0;
            }
        }
        copy_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kBwdRing - 1; ++i) load_next(i);

    int stage = 0;
    int next_row = 0;
    Positions<D> pos;                  // of the warp's next token, loaded a token ahead: under a
                                       // full memory system that takes as long as some passes
    bool on = find(next, next_row);
    if (on) pos.load(A.pos, next_row, A.B, A.T, next.b, next.t, ax, lane);
#pragma unroll 1
    while (on) {
        __syncwarp();                                      // the warp's last unit has read its angles
        token_angles<D>(sh.cs[warp], sh.sn[warp], pos, tab, lane);
        __syncwarp();
        const size_t at_tok = (size_t)next.b * A.T + next.t;
        int ps = next.slice;
        next.step(n_slices, A.T);
        on = find(next, next_row);
        if (on) pos.load(A.pos, next_row, A.B, A.T, next.b, next.t, ax, lane);
        float c[8], s[8];
        lane_angles<D>(sh.cs[warp], sh.sn[warp], j, active, c, s);
        int end = 0, left = 0;
        uint16_t *dst = nullptr;
#pragma unroll 1
        for (; ps < npass; ps += n_slices) {
            const bool value = !QUERIES && ps >= per_kind; // uniform
            if (ps >= end) {
                end = value ? npass : per_kind;
                const int h = (value ? ps - per_kind : ps) * S::kVecPerWarp + slot;
                dst = (QUERIES ? A.dq : value ? A.dv : A.dk) +
                      (at_tok * heads + h) * D + 8 * j;
                left = active ? heads - h : 0;
            }
            copy_wait<kBwdRing - 2>();
            const uint4 *place = &sh.ring[warp][stage][0][lane];
            uint4 ya = make_uint4(0, 0, 0, 0), yb = ya;
            uint4 xa = make_uint4(fill, fill, fill, fill), xb = xa;
            if (left > 0) {
                ya = place[0];
                yb = place[32];
                if (norm && !value) {
                    xa = place[64];
                    xb = place[96];
                }
            }
            load_next(stage == 0 ? kBwdRing - 1 : stage - 1);
            stage = stage == kBwdRing - 1 ? 0 : stage + 1;
            if (!value) backward_vector<D>(xa, xb, ya, yb, c, s, norm, A.eps, gain, dg);
            if (left > 0) {
                *reinterpret_cast<uint4 *>(dst) = ya;
                *reinterpret_cast<uint4 *>(dst + S::kHalf) = yb;
            }
            dst += x_step;
            left -= step_h;
        }
    }
    copy_wait<0>();
    if (!A.partial) return;            // uniform over the grid
    // The lanes of a warp that hold the same coordinates.
#pragma unroll
    for (int e = 0; e < 16; ++e)
#pragma unroll
        for (int x = S::kTPV; x < 32; x <<= 1) dg[e] += __shfl_xor_sync(0xffffffffu, dg[e], x);
    if (slot == 0 && active) {
#pragma unroll
        for (int e = 0; e < 16; ++e) sh.sums[warp][(e < 8 ? 0 : S::kHalf) + 8 * j + (e & 7)] = dg[e];
    }
}

template <int D>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdResident)
norm_rope_backward_kernel(const BackwardArgs A, const __grid_constant__ RopeTable tab,
                          const __grid_constant__ AxisTable ax) {
    __shared__ __align__(16) BackwardShared<D> sh;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // Errors of the sequences.
    for (int b = blockIdx.x * kBwdWarps * 32 + threadIdx.x; b < A.B;
         b += gridDim.x * kBwdWarps * 32) {
        const int p0 = A.pos0 ? A.pos0[b] : 0;
        if (p0 < 0 || (long long)p0 + A.T > A.Lmax)
            report(A.status, p0 < 0 ? GQA_DEV_BAD_LEN : GQA_DEV_CAPACITY);
    }
    if ((int)blockIdx.x < A.n_q)                           // the CTA's role
        backward_units<D, true>(A, tab, ax, sh);
    else
        backward_units<D, false>(A, tab, ax, sh);
    if (!A.partial) return;
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kBwdWarps * 32) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kBwdWarps; ++w) x += sh.sums[w][i];
        A.partial[(size_t)blockIdx.x * D + i] = x;
    }
}

// d gain = the sum of the CTAs' rows (the first n_q: q's, the others: k's): a CTA per 32
// columns of either, 32 rows at a time, added in the order of the rows.
__global__ void __launch_bounds__(1024)
gain_sum_kernel(const float *__restrict__ partial, int n_q, int n_rows, int D, float *dq_gain,
                float *dk_gain) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), r0 = threadIdx.x >> 5;
    float *dst = blockIdx.y == 0 ? dq_gain : dk_gain;
    if (!dst) return;
    const int first = blockIdx.y == 0 ? 0 : n_q, last = blockIdx.y == 0 ? n_q : n_rows;
    float a = 0.f;
    for (int r = first + r0; r < last; r += 32) a += partial[(size_t)r * D + col];
    s[r0][threadIdx.x & 31] = a;
    __syncthreads();
    if (r0 == 0) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
        dst[col] = a;
    }
}

// Slices of a token's passes: one, unless the tokens alone leave most warps idle (64
// single tokens: 4.7 us against 7.2 unsliced; 16384 tokens: 62 us against 77 in two).
int slices(long long tokens, int npass, int warps) {
    const long long want = (warps + tokens - 1) / tokens;
    return (int)(want < 1 ? 1 : want > npass ? npass : want);
}

AxisTable axis_table(const gqa_rope_inputs *x) {
    AxisTable a = {};
    if (x && x->pos)
        for (int i = 0; i < 64; ++i) a.axis[i] = x->pair_axis[i];
    return a;
}

template <int D, bool Q4>
cudaError_t launch_append(AppendArgs A, const gqa_rope_params &p, const gqa_rope_inputs *x,
                          cudaStream_t s) {
    const long long tokens = (long long)A.B * A.T;
    const int per_pass = RopeShape<D>::kVecPerWarp;
    const int npass = ((A.q ? A.Hq : 0) + per_pass - 1) / per_pass +
                      2 * ((A.Hkv + per_pass - 1) / per_pass);
    constexpr int kCtas = 148 * kResident;
    A.n_slices = slices(tokens, npass, kCtas * kWarps);
    const long long ctas = (tokens * A.n_slices + kWarps - 1) / kWarps;
    return launch_pdl(norm_rope_append_kernel<D, Q4>, (unsigned)(ctas < kCtas ? ctas : kCtas),
                      kWarps * 32, s, A, make_table(D, p), axis_table(x));
}

template <int D>
cudaError_t launch_backward(BackwardArgs A, const gqa_rope_params &p, const gqa_rope_inputs *x,
                            float *dq_gain, float *dk_gain, cudaStream_t s) {
    const long long tokens = (long long)A.B * A.T;
    const int per_pass = RopeShape<D>::kVecPerWarp;
    const int npass[2] = {(A.Hq + per_pass - 1) / per_pass,
                          2 * ((A.Hkv + per_pass - 1) / per_pass)};
    // What a token takes in either role, in passes: its angles and the rest of its start
    // about three, a value pass, which is only copied, half a one.
    const double cost[2] = {3.0 + npass[0], 3.0 + 0.75 * npass[1]};
    auto warps_for = [&](int i, int n_ctas) {              // slices, and CTAs that find work
        A.slices[i] = slices(tokens, npass[i], n_ctas * kBwdWarps);
        const long long need = (tokens * A.slices[i] + kBwdWarps - 1) / kBwdWarps;
        return (int)(need < n_ctas ? need : n_ctas);
    };
    // CTAs in that proportion (87 us for 8 x 2048 tokens; by the rows moved 94).  With few
    // tokens a warp the last, partly filled round counts: the best of the shares around it
    // by the longer role's rounds (3 x 1001 tokens: 16.8 us against 18.8).
    const int even = (int)(kBwdMaxCtas * cost[0] / (cost[0] + cost[1]) + 0.5);
    int best = even;
    if (tokens < 16LL * kBwdMaxCtas * kBwdWarps) {
        double least = 1e300;
        for (int n = even - kBwdMaxCtas / 8; n <= even + kBwdMaxCtas / 8; n += 3) {
            if (n < 1 || n >= kBwdMaxCtas) continue;
            double longest = 0;
            for (int i = 0; i < 2; ++i) {
                const long long warps = (long long)(i ? kBwdMaxCtas - n : n) * kBwdWarps;
                const double t = cost[i] * (double)((tokens + warps - 1) / warps);
                longest = t > longest ? t : longest;
            }
            if (longest < least) {
                least = longest;
                best = n;
            }
        }
    }
    best = best < 1 ? 1 : best > kBwdMaxCtas - 1 ? kBwdMaxCtas - 1 : best;
    const int ctas[2] = {warps_for(0, best), warps_for(1, kBwdMaxCtas - best)};
    A.n_q = ctas[0];
    const int grid = ctas[0] + ctas[1];
    cudaError_t e = launch_pdl(norm_rope_backward_kernel<D>, dim3((unsigned)grid), kBwdWarps * 32,
                               s, A, make_table(D, p), axis_table(x));
    if (e != cudaSuccess || !A.partial) return e;
    return launch_pdl(gain_sum_kernel, dim3(D / 32, 2), 1024, s, (const float *)A.partial, A.n_q,
                      grid, D, dq_gain, dk_gain);
}

bool inputs_ok(const gqa_rope_inputs *x, const gqa_rope_params &p, int D) {
    if (!x) return true;
    if ((x->q_gain || x->k_gain) && !p.qk_norm) return false;
    if (!gqa_host::aligned16(x->q_gain) || !gqa_host::aligned16(x->k_gain)) return false;
    if (!x->pos) return true;
    if ((reinterpret_cast<uintptr_t>(x->pos) & 3u) || x->n_axes < 1 || x->n_axes > GQA_MAX_AXES)
        return false;
    for (int i = 0; i < D / 2; ++i)
        if (x->pair_axis[i] >= x->n_axes) return false;
    return true;
}

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks shared by the two appends; the caches are checked by their callers.
gqa_status check_append(const void *q, const void *k, const void *v, const void *q_out,
                        const int32_t *pos0, const int32_t *n_tok, int max_pos0_host,
                        const int32_t *new_len, int B, int T, int Hq, int Hkv, int D, int Lmax,
                        const gqa_rope_params &p, const gqa_rope_inputs *x) {
    using namespace gqa_host;
    if (!k || !v || (q && !q_out) || B < 1 || T < 1 || Hkv < 1 || Lmax < 1)
        return GQA_ERR_INVALID_ARG;
    if (q && (Hq < 1 || Hq % Hkv != 0)) return GQA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        !aligned4(pos0) || !aligned4(n_tok) || !aligned4(new_len))
        return GQA_ERR_INVALID_ARG;
    if (!params_ok(p)) return GQA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return GQA_ERR_UNSUPPORTED;
    if (!inputs_ok(x, p, D)) return GQA_ERR_INVALID_ARG;
    if (Lmax % 128 != 0) return GQA_ERR_INVALID_ARG;
    if ((long long)B * T > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
    // A CTA writes new_len while others still read these, with no order between them.
    auto overlaps = [&](const int32_t *a, long long n) {
        return a && new_len < a + n && a < new_len + B;
    };
    if (new_len && (overlaps(pos0, B) || overlaps(n_tok, B) ||
                    (x && overlaps(x->pos, (long long)x->n_axes * B * T))))
        return GQA_ERR_INVALID_ARG;
    if ((long long)(q ? Hq : 0) + 2LL * Hkv > 0x3fffffffLL) return GQA_ERR_INVALID_ARG;
    if (T > Lmax && !n_tok) return GQA_ERR_CAPACITY;
    if (max_pos0_host >= 0 && !n_tok && (long long)max_pos0_host + T > Lmax)
        return GQA_ERR_CAPACITY;
    if (max_pos0_host > Lmax) return GQA_ERR_CAPACITY;
    return GQA_OK;
}

AppendArgs append_args(const void *q, const void *k, const void *v, void *q_out,
                       const int32_t *pos0, const int32_t *n_tok, int32_t *new_len, int B, int T,
                       int Hq, int Hkv, int Lmax, const gqa_rope_params &p,
                       const gqa_rope_inputs *x, int32_t *status) {
    AppendArgs A = {};
    A.q = static_cast<const uint16_t *>(q);
    A.k = static_cast<const uint16_t *>(k);
    A.v = static_cast<const uint16_t *>(v);
    A.q_out = static_cast<uint16_t *>(q_out);
    A.pos0 = pos0;
    A.n_tok = n_tok;
    A.new_len = new_len;
    A.status = status;
    A.B = B;
    A.T = T;
    A.Hq = Hq;
    A.Hkv = Hkv;
    A.Lmax = Lmax;
    A.qk_norm = p.qk_norm;
    A.eps = p.eps;
    if (x) {
        A.q_gain = static_cast<const uint16_t *>(x->q_gain);
        A.k_gain = static_cast<const uint16_t *>(x->k_gain);
        A.pos = x->pos;
    }
    return A;
}

}  // namespace
}  // namespace gqa

extern "C" gqa_status gqa_norm_rope_append(const void *q, const void *k, const void *v,
                                           void *q_out, void *k_cache, void *v_cache,
                                           const int32_t *pos0, const int32_t *n_tok,
                                           int max_pos0_host, int32_t *new_len, int B, int T,
                                           int Hq, int Hkv, int D, int Lmax, gqa_rope_params p,
                                           const gqa_rope_inputs *x, int32_t *status_dev,
                                           void *stream) {
    using namespace gqa_host;
    if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache))
        return GQA_ERR_INVALID_ARG;
    const gqa_status st = gqa::check_append(q, k, v, q_out, pos0, n_tok, max_pos0_host, new_len,
                                            B, T, Hq, Hkv, D, Lmax, p, x);
    if (st != GQA_OK) return st;
    gqa::AppendArgs A = gqa::append_args(q, k, v, q_out, pos0, n_tok, new_len, B, T, Hq, Hkv,
                                         Lmax, p, x, status_dev);
    A.kc = static_cast<uint16_t *>(k_cache);
    A.vc = static_cast<uint16_t *>(v_cache);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 64   ? gqa::launch_append<64, false>(A, p, x, s)
                          : D == 96 ? gqa::launch_append<96, false>(A, p, x, s)
                                    : gqa::launch_append<128, false>(A, p, x, s);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

extern "C" gqa_status gqa_norm_rope_append_q4(const void *q, const void *k, const void *v,
                                              void *q_out, void *k_codes, void *k_scales,
                                              void *v_codes, void *v_scales, const int32_t *pos0,
                                              const int32_t *n_tok, int max_pos0_host,
                                              int32_t *new_len, int B, int T, int Hq, int Hkv,
                                              int D, int Lmax, gqa_rope_params p,
                                              const gqa_rope_inputs *x, int32_t *status_dev,
                                              void *stream) {
    using namespace gqa_host;
    if (!k_codes || !k_scales || !v_codes || !v_scales || !aligned16(k_codes) ||
        !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales))
        return GQA_ERR_INVALID_ARG;
    const gqa_status st = gqa::check_append(q, k, v, q_out, pos0, n_tok, max_pos0_host, new_len,
                                            B, T, Hq, Hkv, D, Lmax, p, x);
    if (st != GQA_OK) return st;
    gqa::AppendArgs A = gqa::append_args(q, k, v, q_out, pos0, n_tok, new_len, B, T, Hq, Hkv,
                                         Lmax, p, x, status_dev);
    A.k_codes = static_cast<uint8_t *>(k_codes);
    A.v_codes = static_cast<uint8_t *>(v_codes);
    A.k_scales = static_cast<uint32_t *>(k_scales);
    A.v_scales = static_cast<uint32_t *>(v_scales);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 64   ? gqa::launch_append<64, true>(A, p, x, s)
                          : D == 96 ? gqa::launch_append<96, true>(A, p, x, s)
                                    : gqa::launch_append<128, true>(A, p, x, s);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

extern "C" size_t gqa_norm_rope_backward_workspace_bytes(int D) {
    return gqa_host::head_dim_ok(D) ? (size_t)gqa::kBwdMaxCtas * D * 4 : 0;
}

extern "C" gqa_status gqa_norm_rope_append_backward(
    const void *q, const void *k, const void *dq_out, const void *dk_cache, const void *dv_cache,
    void *dq, void *dk, void *dv, float *dq_gain, float *dk_gain, const int32_t *pos0,
    int max_pos0_host, int B, int T, int Hq, int Hkv, int D, int Lmax, gqa_rope_params p,
    const gqa_rope_inputs *x, void *ws, size_t ws_bytes, int32_t *status_dev, void *stream) {
    using namespace gqa_host;
    if (!q || !k || !dq_out || !dk_cache || !dv_cache || !dq || !dk || !dv || B < 1 || T < 1 ||
        Hq < 1 || Hkv < 1 || Lmax < 1 || Hq % Hkv != 0)
        return GQA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(dq_out) || !aligned16(dk_cache) ||
        !aligned16(dv_cache) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
        !gqa::aligned4(dq_gain) || !gqa::aligned4(dk_gain) || !gqa::aligned4(pos0))
        return GQA_ERR_INVALID_ARG;
    if (!gqa::params_ok(p) || ((dq_gain || dk_gain) && !p.qk_norm)) return GQA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return GQA_ERR_UNSUPPORTED;
    if (!gqa::inputs_ok(x, p, D)) return GQA_ERR_INVALID_ARG;
    if (Lmax % 128 != 0) return GQA_ERR_INVALID_ARG;
    if ((long long)B * T > 0x7fffffffLL || (long long)Hq + 2LL * Hkv > 0x3fffffffLL)
        return GQA_ERR_INVALID_ARG;
    if (T > Lmax || (max_pos0_host >= 0 && (long long)max_pos0_host + T > Lmax))
        return GQA_ERR_CAPACITY;
    const bool gains = dq_gain || dk_gain;
    if (gains && (!ws || !aligned16(ws) || ws_bytes < gqa_norm_rope_backward_workspace_bytes(D)))
        return GQA_ERR_WORKSPACE;
    gqa::BackwardArgs A = {};
    A.q = static_cast<const uint16_t *>(q);
    A.k = static_cast<const uint16_t *>(k);
    A.dq_out = static_cast<const uint16_t *>(dq_out);
    A.dkc = static_cast<const uint16_t *>(dk_cache);
    A.dvc = static_cast<const uint16_t *>(dv_cache);
    A.dq = static_cast<uint16_t *>(dq);
    A.dk = static_cast<uint16_t *>(dk);
    A.dv = static_cast<uint16_t *>(dv);
    A.pos0 = pos0;
    A.partial = gains ? static_cast<float *>(ws) : nullptr;
    A.status = status_dev;
    A.B = B;
    A.T = T;
    A.Hq = Hq;
    A.Hkv = Hkv;
    A.Lmax = Lmax;
    A.qk_norm = p.qk_norm;
    A.eps = p.eps;
    if (x) {
        A.q_gain = static_cast<const uint16_t *>(x->q_gain);
        A.k_gain = static_cast<const uint16_t *>(x->k_gain);
        A.pos = x->pos;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 64   ? gqa::launch_backward<64>(A, p, x, dq_gain, dk_gain, s)
                          : D == 96 ? gqa::launch_backward<96>(A, p, x, dq_gain, dk_gain, s)
                                    : gqa::launch_backward<128>(A, p, x, dq_gain, dk_gain, s);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}
