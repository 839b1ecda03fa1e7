// norm_rope.cu -- per-head RMSNorm with learned gains, rotation by positions on up
// to four axes, and the write into a bf16 or a 4-bit cache, in one pass; and the
// backward of the bf16 form.
//
//   u = gain * x * (mean x^2 + eps)^(-1/2),   y = mscale * R(P) u,
//   pair i (coordinates i, i + D/2) turned by P_i theta_i, P_i the token's position
//   on pair i's axis (image and video tokens: time, height, width).
//
// Forward.  Bound by memory: q is read and written once, k and v read once, the
// cache rows written once.  A warp takes one token (or, when there are few tokens,
// one slice of a token's vectors, so that a decode step still spreads over the
// SMs); it walks the token's Hq query, Hkv key and Hkv value vectors kVecPerWarp at
// a time, kAhead passes loaded before any is used, the first ones before the angles
// are computed.  A vector is held by 4 or 8 lanes, lane j with coordinates
// 8j .. 8j+7 and D/2 + 8j ..: both members of its 8 rotation pairs, and half of one
// group of the 4-bit row, so rotation needs no exchange, the norm one shuffle sum
// and the quantiser one shuffle per group.
#include "q4.cuh"
#include "rope.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 4;              // warps per CTA
constexpr int kAhead = 5;              // passes loaded ahead
constexpr int kWantWarps = 148 * 16;   // warps that fill the device

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
    int B, T, Hq, Hkv, Lmax, n_slices;
    int qk_norm;
    float eps;
};

// cos / sin of the token's D/2 angles into the warp's rows: position times theta_i
// in float64, reduced to [-pi, pi] in float64, then fp32.
template <int D>
__device__ __forceinline__ void token_angles(float *cs, float *sn, const int32_t *pos, int p_seq,
                                             int B, int T, int b, int t, const RopeTable &tab,
                                             const AxisTable &ax, int lane) {
#pragma unroll
    for (int i = lane; i < D / 2; i += 32) {
        const int p = pos ? pos[((size_t)ax.axis[i] * B + b) * T + t] : p_seq;
        const double a = (double)p * tab.theta[i];
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

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32)
norm_rope_append_kernel(const AppendArgs A, const __grid_constant__ RopeTable tab,
                        const __grid_constant__ AxisTable ax) {
    using S = RopeShape<D>;
    using R = Q4Shape<D>;
    __shared__ __align__(16) float cs[kWarps][S::kHalf];
    __shared__ __align__(16) float sn[kWarps][S::kHalf];
    __shared__ __align__(16) float gain[2][D];
    // A programmatic dependent of the kernel before it, which may have produced any
    // of its inputs: wait for that kernel to complete before reading.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    load_gains<D>(gain, A.q_gain, A.k_gain, threadIdx.x, kWarps * 32);
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * kWarps + warp;
    const int tok = (int)(unit / A.n_slices);
    const int slice = (int)(unit - (long long)tok * A.n_slices);
    if (tok >= A.B * A.T) return;                  // only warp-level sync follows
    const int b = tok / A.T, t = tok - b * A.T;
    const int p0 = A.pos0 ? A.pos0[b] : 0;
    const int n = A.n_tok ? A.n_tok[b] : A.T;
    const bool bad = p0 < 0 || n < 0 || n > A.T;
    const long long end = (long long)p0 + (bad ? 0 : n);
    if (t == 0 && slice == 0 && lane == 0) {
        if (bad) report(A.status, GQA_DEV_BAD_LEN);
        else if (end > A.Lmax) report(A.status, GQA_DEV_CAPACITY);
        if (A.new_len) A.new_len[b] = (int)(end < 0x7fffffffLL ? end : 0x7fffffffLL);
    }
    if (bad || end > A.Lmax || t >= n) return;
    const int slot_row = p0 + t;

    const int j = lane % S::kTPV;
    const int slot = lane / S::kTPV;
    const bool active = j < S::kChunks;
    const int nq = A.q ? A.Hq : 0, nk = A.Hkv;
    const int nrot = nq + nk, nvec = nrot + nk;
    const int npass = (nvec + S::kVecPerWarp - 1) / S::kVecPerWarp;

    auto source = [&](int r) -> const uint16_t * {
        if (r < nq) return A.q + ((size_t)tok * A.Hq + r) * D;
        if (r < nrot) return A.k + ((size_t)tok * A.Hkv + (r - nq)) * D;
        return A.v + ((size_t)tok * A.Hkv + (r - nrot)) * D;
    };

    float c[8], sv[8];
    const int step = A.n_slices;
    for (int pb = slice; pb < npass; pb += step * kAhead) {
        uint4 ra[kAhead], rb[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = (pb + u * step) * S::kVecPerWarp + slot;
            ra[u] = make_uint4(0, 0, 0, 0);
            rb[u] = make_uint4(0, 0, 0, 0);
            if (r < nvec && active) {
                const uint16_t *src = source(r);
                ra[u] = *reinterpret_cast<const uint4 *>(src + 8 * j);
                rb[u] = *reinterpret_cast<const uint4 *>(src + S::kHalf + 8 * j);
            }
        }
        if (pb == slice) {
            token_angles<D>(cs[warp], sn[warp], A.pos, slot_row, A.B, A.T, b, t, tab, ax, lane);
            __syncwarp();
            lane_angles<D>(cs[warp], sn[warp], j, active, c, sv);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (pb + u * step >= npass) break;             // uniform across the warp
            const int r0 = (pb + u * step) * S::kVecPerWarp;
            const int r = r0 + slot;
            const bool mem = r < nvec && active;
            uint4 a = ra[u], bb = rb[u];
            if (r0 < nrot) {                               // uniform across the warp
                uint4 oa, ob;
                rotate_vector<D, true>(a, bb, oa, ob, c, sv, mem, A.qk_norm != 0, A.eps,
                                       gain[r < nq ? 0 : 1] + 8 * j);
                if (r < nrot) {
                    a = oa;
                    bb = ob;
                }
            }
            if constexpr (!Q4) {
                if (mem) {
                    uint16_t *dst;
                    if (r < nq) {
                        dst = A.q_out + ((size_t)tok * A.Hq + r) * D;
                    } else {
                        const int h = r < nrot ? r - nq : r - nrot;
                        dst = (r < nrot ? A.kc : A.vc) +
                              (((size_t)b * A.Hkv + h) * A.Lmax + slot_row) * D;
                    }
                    *reinterpret_cast<uint4 *>(dst + 8 * j) = a;
                    *reinterpret_cast<uint4 *>(dst + S::kHalf + 8 * j) = bb;
                }
            } else {
                if (mem && r < nq) {
                    uint16_t *dst = A.q_out + ((size_t)tok * A.Hq + r) * D;
                    *reinterpret_cast<uint4 *>(dst + 8 * j) = a;
                    *reinterpret_cast<uint4 *>(dst + S::kHalf + 8 * j) = bb;
                }
                if (r0 + S::kVecPerWarp > nq) {            // uniform: some vector is K or V
                    uint32_t codes[2], sm;
                    q4_quantise(a, bb, codes, sm);
                    if (mem && r >= nq) {
                        const int h = r < nrot ? r - nq : r - nrot;
                        const size_t row = ((size_t)b * A.Hkv + h) * A.Lmax + slot_row;
                        const int g = j >> 1, k0 = 2 * (j & 1);
                        uint32_t *cw = reinterpret_cast<uint32_t *>(r < nrot ? A.k_codes
                                                                             : A.v_codes) +
                                       row * (R::kCodeBytes / 4);
                        cw[R::NG * k0 + g] = codes[0];
                        cw[R::NG * (k0 + 1) + g] = codes[1];
                        if ((j & 1) == 0) (r < nrot ? A.k_scales : A.v_scales)[row * R::NG + g] = sm;
                    }
                }
            }
        }
    }
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
// Bound by memory: x, dy read once and dx written once.  Warps take (token, slice)
// units as in the forward, a fixed number of them in turn, and keep the sums of
// d gain for their lanes' 16 coordinates in registers over all their units; a CTA
// adds its warps' sums and leaves one row per CTA in the workspace, and a second
// kernel adds the rows in a fixed order, so equal calls give equal bits.
constexpr int kBwdWarps = 8;
constexpr int kBwdMaxCtas = 2 * 148;   // two CTAs per SM
constexpr int kBwdAhead = 2;           // passes loaded ahead (two vectors each)

struct BackwardArgs {
    const uint16_t *q, *k, *dq_out, *dkc, *dvc;
    uint16_t *dq, *dk, *dv;
    const uint16_t *q_gain, *k_gain;
    const int32_t *pos0, *pos;
    float *partial;                    // [CTAs][2][D], NULL: no gain gradients wanted
    int32_t *status;
    int B, T, Hq, Hkv, Lmax, n_slices;
    int qk_norm;
    float eps;
};

// One vector: dx of the lane's 16 coordinates, and its share of d gain added to dg.
template <int D>
__device__ __forceinline__ void backward_vector(const uint4 xa_in, const uint4 xb_in,
                                                const uint4 ya_in, const uint4 yb_in, uint4 &da,
                                                uint4 &db, const float (&c)[8],
                                                const float (&sv)[8], bool live, bool qk_norm,
                                                float eps, const float *gain, float (&dg)[16]) {
    using S = RopeShape<D>;
    const uint32_t xw[8] = {xa_in.x, xa_in.y, xa_in.z, xa_in.w,
                            xb_in.x, xb_in.y, xb_in.z, xb_in.w};
    const uint32_t yw[8] = {ya_in.x, ya_in.y, ya_in.z, ya_in.w,
                            yb_in.x, yb_in.y, yb_in.z, yb_in.w};
    float w[16];                       // [0..7] first-half chunk, [8..15] second-half chunk
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float a0 = bf16lo(yw[e]), a1 = bf16hi(yw[e]);
        const float b0 = bf16lo(yw[4 + e]), b1 = bf16hi(yw[4 + e]);
        const float c0 = c[2 * e], c1 = c[2 * e + 1], s0 = sv[2 * e], s1 = sv[2 * e + 1];
        mul2(w[2 * e], w[2 * e + 1], b0, b1, s0, s1);
        fma2(w[2 * e], w[2 * e + 1], a0, a1, c0, c1, w[2 * e], w[2 * e + 1]);
        mul2(w[8 + 2 * e], w[9 + 2 * e], a0, a1, -s0, -s1);
        fma2(w[8 + 2 * e], w[9 + 2 * e], b0, b1, c0, c1, w[8 + 2 * e], w[9 + 2 * e]);
    }
    if (qk_norm) {                     // uniform
        float ss0 = 0.f, ss1 = 0.f, xz0 = 0.f, xz1 = 0.f;
        float z[16];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x0 = bf16lo(xw[e]), x1 = bf16hi(xw[e]);
            float g0 = 0.f, g1 = 0.f;
            if (live) {
                const float2 gg = *reinterpret_cast<const float2 *>(
                    gain + (e < 4 ? 2 * e : S::kHalf + 2 * (e - 4)));
                g0 = gg.x;
                g1 = gg.y;
            }
            fma2(ss0, ss1, x0, x1, x0, x1, ss0, ss1);
            mul2(z[2 * e], z[2 * e + 1], w[2 * e], w[2 * e + 1], g0, g1);
            fma2(xz0, xz1, x0, x1, z[2 * e], z[2 * e + 1], xz0, xz1);
        }
        const float ss = group_sum<S::kTPV>(ss0 + ss1);      // lanes not live hold zeros
        const float xz = group_sum<S::kTPV>(xz0 + xz1);
        const float r = live ? rsqrtf(ss * (1.0f / D) + eps) : 0.f;
        const float k = -r * (xz * r * (1.0f / D));          // r^3 alone could overflow
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x0 = bf16lo(xw[e]), x1 = bf16hi(xw[e]);
            float t0, t1;
            mul2(t0, t1, x0, x1, r, r);
            fma2(dg[2 * e], dg[2 * e + 1], w[2 * e], w[2 * e + 1], t0, t1, dg[2 * e],
                 dg[2 * e + 1]);
            mul2(t0, t1, t0, t1, k, k);
            fma2(w[2 * e], w[2 * e + 1], z[2 * e], z[2 * e + 1], r, r, t0, t1);
        }
    }
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = pack_bf16x2(w[2 * e], w[2 * e + 1]);
    da = make_uint4(o[0], o[1], o[2], o[3]);
    db = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D>
__global__ void __launch_bounds__(kBwdWarps * 32, 2)
norm_rope_backward_kernel(const BackwardArgs A, const __grid_constant__ RopeTable tab,
                          const __grid_constant__ AxisTable ax) {
    using S = RopeShape<D>;
    __shared__ __align__(16) float cs[kBwdWarps][S::kHalf];
    __shared__ __align__(16) float sn[kBwdWarps][S::kHalf];
    __shared__ __align__(16) float gain[2][D];
    __shared__ __align__(16) float sums[kBwdWarps][2][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    load_gains<D>(gain, A.q_gain, A.k_gain, threadIdx.x, kBwdWarps * 32);
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int j = lane % S::kTPV, slot = lane / S::kTPV;
    const bool active = j < S::kChunks;
    // Passes of one kind each: query heads, then key heads, then value heads.
    const int qp = (A.Hq + S::kVecPerWarp - 1) / S::kVecPerWarp;
    const int kp = (A.Hkv + S::kVecPerWarp - 1) / S::kVecPerWarp;
    const int npass = qp + 2 * kp;
    float dgq[16], dgk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) dgq[e] = dgk[e] = 0.f;

    const long long units = (long long)A.B * A.T * A.n_slices;
    const long long stride = (long long)gridDim.x * kBwdWarps;
    for (long long unit = (long long)blockIdx.x * kBwdWarps + warp; unit < units;
         unit += stride) {
        const int tok = (int)(unit / A.n_slices);
        const int slice = (int)(unit - (long long)tok * A.n_slices);
        const int b = tok / A.T, t = tok - b * A.T;
        const int p0 = A.pos0 ? A.pos0[b] : 0;
        if (p0 < 0 || (long long)p0 + A.T > A.Lmax) {
            if (t == 0 && slice == 0 && lane == 0)
                report(A.status, p0 < 0 ? GQA_DEV_BAD_LEN : GQA_DEV_CAPACITY);
            continue;
        }
        const int slot_row = p0 + t;
        float c[8], sv[8];
        for (int pb = slice; pb < npass; pb += A.n_slices * kBwdAhead) {
            uint4 x[kBwdAhead][2], y[kBwdAhead][2];
#pragma unroll
            for (int u = 0; u < kBwdAhead; ++u) {
                const int ps = pb + u * A.n_slices;
                const bool is_q = ps < qp, is_k = !is_q && ps < qp + kp;
                const int h = (is_q ? ps : is_k ? ps - qp : ps - qp - kp) * S::kVecPerWarp + slot;
                x[u][0] = x[u][1] = y[u][0] = y[u][1] = make_uint4(0, 0, 0, 0);
                if (ps < npass && active && h < (is_q ? A.Hq : A.Hkv)) {
                    const size_t in = is_q ? ((size_t)tok * A.Hq + h) * D
                                           : ((size_t)tok * A.Hkv + h) * D;
                    const size_t row = (((size_t)b * A.Hkv + h) * A.Lmax + slot_row) * D;
                    const uint16_t *ys = is_q ? A.dq_out + in : (is_k ? A.dkc : A.dvc) + row;
                    y[u][0] = *reinterpret_cast<const uint4 *>(ys + 8 * j);
                    y[u][1] = *reinterpret_cast<const uint4 *>(ys + S::kHalf + 8 * j);
                    if ((is_q || is_k) && A.qk_norm) {
                        const uint16_t *xs = (is_q ? A.q : A.k) + in;
                        x[u][0] = *reinterpret_cast<const uint4 *>(xs + 8 * j);
                        x[u][1] = *reinterpret_cast<const uint4 *>(xs + S::kHalf + 8 * j);
                    }
                }
            }
            if (pb == slice) {
                __syncwarp();          // the warp's last unit has read its angles
                token_angles<D>(cs[warp], sn[warp], A.pos, slot_row, A.B, A.T, b, t, tab, ax,
                                lane);
                __syncwarp();
                lane_angles<D>(cs[warp], sn[warp], j, active, c, sv);
            }
#pragma unroll
            for (int u = 0; u < kBwdAhead; ++u) {
                const int ps = pb + u * A.n_slices;
                if (ps >= npass) break;                    // uniform across the warp
                const bool is_q = ps < qp, is_k = !is_q && ps < qp + kp;
                const int h = (is_q ? ps : is_k ? ps - qp : ps - qp - kp) * S::kVecPerWarp + slot;
                const bool live = active && h < (is_q ? A.Hq : A.Hkv);
                uint4 da = y[u][0], db = y[u][1];
                if (is_q)
                    backward_vector<D>(x[u][0], x[u][1], y[u][0], y[u][1], da, db, c, sv, live,
                                       A.qk_norm != 0, A.eps, gain[0] + 8 * j, dgq);
                else if (is_k)
                    backward_vector<D>(x[u][0], x[u][1], y[u][0], y[u][1], da, db, c, sv, live,
                                       A.qk_norm != 0, A.eps, gain[1] + 8 * j, dgk);
                if (live) {
                    uint16_t *dst = is_q ? A.dq + ((size_t)tok * A.Hq + h) * D
                                         : (is_k ? A.dk : A.dv) + ((size_t)tok * A.Hkv + h) * D;
                    *reinterpret_cast<uint4 *>(dst + 8 * j) = da;
                    *reinterpret_cast<uint4 *>(dst + S::kHalf + 8 * j) = db;
                }
            }
        }
    }
    if (!A.partial) return;            // uniform over the grid
    // The lanes of a warp that hold the same coordinates, then the CTA's warps.
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
        for (int o = S::kTPV; o < 32; o <<= 1) {
            dgq[e] += __shfl_xor_sync(0xffffffffu, dgq[e], o);
            dgk[e] += __shfl_xor_sync(0xffffffffu, dgk[e], o);
        }
    }
    if (slot == 0 && active) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int d = (e < 8 ? 0 : S::kHalf) + 8 * j + (e & 7);
            sums[warp][0][d] = dgq[e];
            sums[warp][1][d] = dgk[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += kBwdWarps * 32) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kBwdWarps; ++w) s += sums[w][i / D][i % D];
        A.partial[(size_t)blockIdx.x * 2 * D + i] = s;
    }
}

// d gain = the sum of the CTAs' rows: a CTA per 32 of the 2 D columns, 32 rows at a
// time, added in the order of the rows.
__global__ void __launch_bounds__(1024)
gain_sum_kernel(const float *__restrict__ partial, int n_rows, int D, float *dq_gain,
                float *dk_gain) {
    __shared__ float s[32][33];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), r0 = threadIdx.x >> 5;
    float a = 0.f;
    for (int r = r0; r < n_rows; r += 32) a += partial[(size_t)r * 2 * D + col];
    s[r0][threadIdx.x & 31] = a;
    __syncthreads();
    if (r0 == 0) {
        a = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) a += s[i][threadIdx.x];
        float *dst = col < D ? dq_gain : dk_gain;
        if (dst) dst[col < D ? col : col - D] = a;
    }
}

// Slices of a token's passes: one, unless the tokens alone leave most warps idle.
int slices(long long tokens, int npass) {
    const long long want = (kWantWarps + tokens - 1) / tokens;
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
    A.n_slices = slices(tokens, ((A.q ? A.Hq : 0) + 2 * A.Hkv + per_pass - 1) / per_pass);
    const long long ctas = (tokens * A.n_slices + kWarps - 1) / kWarps;
    return launch_pdl(norm_rope_append_kernel<D, Q4>, (unsigned)ctas, kWarps * 32, s, A,
                      make_table(D, p), axis_table(x));
}

template <int D>
cudaError_t launch_backward(BackwardArgs A, const gqa_rope_params &p, const gqa_rope_inputs *x,
                            float *dq_gain, float *dk_gain, cudaStream_t s) {
    const long long tokens = (long long)A.B * A.T;
    const int per_pass = RopeShape<D>::kVecPerWarp;
    A.n_slices = slices(tokens, (A.Hq + per_pass - 1) / per_pass +
                                    2 * ((A.Hkv + per_pass - 1) / per_pass));
    const long long ctas = (tokens * A.n_slices + kBwdWarps - 1) / kBwdWarps;
    const unsigned grid = (unsigned)(ctas < kBwdMaxCtas ? ctas : kBwdMaxCtas);
    cudaError_t e = launch_pdl(norm_rope_backward_kernel<D>, grid, kBwdWarps * 32, s, A,
                               make_table(D, p), axis_table(x));
    if (e != cudaSuccess || !A.partial) return e;
    return launch_pdl(gain_sum_kernel, 2 * D / 32, 1024, s, (const float *)A.partial, (int)grid,
                      D, dq_gain, dk_gain);
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
    if (new_len && (new_len == pos0 || new_len == n_tok)) return GQA_ERR_INVALID_ARG;
    if (!params_ok(p)) return GQA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return GQA_ERR_UNSUPPORTED;
    if (!inputs_ok(x, p, D)) return GQA_ERR_INVALID_ARG;
    if (Lmax % 128 != 0) return GQA_ERR_INVALID_ARG;
    if ((long long)B * T > 0x7fffffffLL) return GQA_ERR_INVALID_ARG;
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
    return gqa_host::head_dim_ok(D) ? (size_t)gqa::kBwdMaxCtas * 2 * D * 4 : 0;
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
