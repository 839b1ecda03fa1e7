// decode_q4.cu -- single-token attention against a cache held in 4 bits, and the
// read-back of such a cache as bf16.
//
//   out[b,h,:] = sum_{s < lens[b]} softmax_s(q[b,h,:] . K[b,h/g,s,:] scale) V[b,h/g,s,:]
// with K and V the values m + s c of the rows (q4.cuh), never rounded to bf16.
//
// A token of one KV head is D/2 + D/8 bytes each for K and V (160 bytes together
// at D = 128, against 512 in bf16): at full memory rate an SM receives some 45
// codes per clock, three query heads make that 135 multiply-adds per clock, and
// each code has to be unpacked first; scalar arithmetic cannot keep up, so the
// products run on the tensor cores with the codes as they are:
//   * (w & 0x000f000f) | 0x43004300 turns two codes of a word into the bf16 pair
//     128 + c, exactly, in one instruction.  Codes are the 16-row operand of
//     mma.m16n8k16 (rows = keys for the scores, coordinates for the output) and the
//     query heads its 8 columns: a group of heads costs what one head costs.
//   * scores: q is bf16 already, so the products are exact; a group's sum a is
//     scaled and shifted once: s a + (m - 128 s) sum(q) over the group.
//   * output: sum_k p_k (m_k + s_k c_k,d).  p_k s_k goes in as the 8-column operand,
//     carried by movmatrix from the score layout.  Rounded to bf16 it would cost
//     2^-9 per term, so it goes in twice, as a rounded part and the bf16 of what the
//     rounding left (2^-17 together): with up to 4 heads per CTA the second part
//     uses columns 4 .. 7 (q is repeated there, so those lanes hold the same p),
//     with 5 .. 8 a second mma.  The 128 in every code is taken out by a column sum
//     of the same operand, 128 sum(p s), from one more mma; sum(p m) is added up in
//     fp32 beside it.
// mma.sync rather than tcgen05: its operands come from registers, where the codes
// are unpacked; tcgen05 would need them written to shared memory as bf16, four
// times the bytes that arrived, for 8 columns of work.
//
// Work: as decode.cu, one CTA per (chunk of 64 NT cache slots, KV head x head
// subgroup, sequence), its loads four bulk copies (K codes and scales with q on one
// barrier, V's on another), its four warps taking 16-key tiles in turn; statistics
// and partial outputs are merged in shared memory, the chunk's (m, l, o) goes to
// the workspace and a second kernel, a programmatic dependent, merges the chunks.
// When one chunk covers max_len the CTA writes the output itself.
#include "q4.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = 8;               // columns of the mma: query heads of a CTA, at most

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values spread over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Codes at bits 0 and 16 of w >> sh as the bf16 pair 128 + c.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int sh) {
    return ((w >> sh) & 0x000f000fu) | 0x43004300u;
}

template <int NG>
__device__ __forceinline__ void load_words(uint32_t (&w)[NG], const uint32_t *p) {
    if constexpr (NG == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (NG == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < NG; ++i) w[i] = p[i];
    }
}

template <int D, int NT>
struct DecQ4Shape {
    static constexpr int NG = Q4Shape<D>::NG;
    static constexpr int CH = 64 * NT;                     // cache slots per CTA
    static constexpr int kRowWords = D / 8;                // 4-byte words of codes per row
    static constexpr int kCode = CH * D / 2;
    static constexpr int kScale = CH * 4 * NG;
    // [K codes][K scales][V codes][V scales] | [q][(m, l)]; the warps' partial
    // outputs (kWarps x kCols x (D + 4) f32) are written over the first part once
    // every warp is done with it.  D + 4: the four lanes of a row write four columns,
    // 8 banks apart.
    static constexpr int kOffKS = kCode;
    static constexpr int kOffV = kCode + kScale;
    static constexpr int kOffVS = kOffV + kCode;
    static constexpr int kPartStride = D + 4;
    static constexpr int kPart = kWarps * kCols * kPartStride * 4;
    static constexpr int kData = kOffVS + kScale;
    static constexpr int kOffQ = (kData > kPart ? kData : kPart) + 0;
    static constexpr int kOffML = kOffQ + kCols * D * 2;
    static constexpr int kSmem = kOffML + kWarps * kCols * 2 * 4;
    static_assert(kOffQ % 16 == 0 && kOffV % 16 == 0 && kOffVS % 16 == 0, "alignment");
};

struct DecQ4Args {
    const uint16_t *q;
    const uint8_t *kc, *vc;
    const uint32_t *ks, *vs;
    const int32_t *lens;
    uint16_t *out;
    float *ws_ml, *ws_o;
    int32_t *status;
    int max_len, B, Hq, Hkv, Lmax, n_splits, n_sub, G;   // G: query heads per CTA
    float scale_log2;
};

// Workspace: [(m, l): rows x 2 f32][o: rows x D f32], rows = B x Hq x n_splits, row
// (b, h, c) = (b * Hq + h) * n_splits + c.  WIDE: 5 .. 8 query heads per CTA.
template <int D, int NT, bool WIDE>
__global__ void __launch_bounds__(kThreads, 4)
decode_q4_kernel(const DecQ4Args A) {
    using S = DecQ4Shape<D, NT>;
    constexpr int NG = S::NG;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[2];              // [0]: K and q, [1]: V
    __shared__ float sw[kWarps * kCols];                   // merge weights [warp][column]
    __shared__ float s_inv[kCols];

    // Wait for the kernel before this one (normally the append that wrote lens and
    // the newest slot) before reading; the merge may then be scheduled.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int c = blockIdx.x;
    const int kvh = blockIdx.y / A.n_sub, sub = blockIdx.y - kvh * A.n_sub;
    const int b = blockIdx.z;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = A.Hq / A.Hkv;
    const int h0 = kvh * group + sub * A.G;                // first query head
    const int G = min(A.G, group - sub * A.G);             // query heads of this CTA
    const int len = A.lens[b];
    if (len < 1 || len > A.max_len || len > A.Lmax) {
        if (c == 0 && blockIdx.y == 0 && tid == 0)
            report(A.status, len < 1 ? GQA_DEV_BAD_LEN : GQA_DEV_CAPACITY);
        if (A.n_splits == 1)
            for (int i = tid; i < G * D; i += kThreads) A.out[((size_t)b * A.Hq + h0) * D + i] = 0;
        return;
    }
    const int key0 = c * S::CH;
    if (key0 >= len) return;
    const int nk = min(S::CH, len - key0);
    const uint32_t bar_k = ptx::smem_addr(&bars[0]);
    const uint32_t bar_v = ptx::smem_addr(&bars[1]);
    if (tid == 0) {
        ptx::mbar_init(bar_k, 1);
        ptx::mbar_init(bar_v, 1);
        ptx::fence_barrier_init();
        // Whole groups of 4 rows: a row's scales may be 8 or 12 bytes and a bulk copy
        // moves multiples of 16.  Lmax is a multiple of 128, so the rows exist.
        const int nr = (nk + 3) & ~3;
        const uint32_t cb = (uint32_t)nr * (D / 2), sb = (uint32_t)nr * (4 * NG);
        const size_t row = ((size_t)b * A.Hkv + kvh) * A.Lmax + key0;
        const uint64_t pol = ptx::policy_evict_first();
        ptx::mbar_arrive_expect_tx(bar_k, cb + sb + G * D * 2);
        ptx::bulk_g2s(ptx::smem_addr(smem + S::kOffQ), A.q + ((size_t)b * A.Hq + h0) * D,
                      G * D * 2, bar_k);
        ptx::bulk_g2s_hint(ptx::smem_addr(smem), A.kc + row * (D / 2), cb, bar_k, pol);
        ptx::bulk_g2s_hint(ptx::smem_addr(smem + S::kOffKS), A.ks + row * NG, sb, bar_k, pol);
        ptx::mbar_arrive_expect_tx(bar_v, cb + sb);
        ptx::bulk_g2s_hint(ptx::smem_addr(smem + S::kOffV), A.vc + row * (D / 2), cb, bar_v, pol);
        ptx::bulk_g2s_hint(ptx::smem_addr(smem + S::kOffVS), A.vs + row * NG, sb, bar_v, pol);
    }
    __syncthreads();                   // barriers initialised before anyone waits on them
    const uint32_t *kw = reinterpret_cast<const uint32_t *>(smem);
    const uint32_t *ksw = reinterpret_cast<const uint32_t *>(smem + S::kOffKS);
    const uint32_t *vw = reinterpret_cast<const uint32_t *>(smem + S::kOffV);
    const uint32_t *vsw = reinterpret_cast<const uint32_t *>(smem + S::kOffVS);
    const uint16_t *qs = reinterpret_cast<const uint16_t *>(smem + S::kOffQ);
    float *wml = reinterpret_cast<float *>(smem + S::kOffML);        // [warp][column][2]
    float *part = reinterpret_cast<float *>(smem);                   // [warp][column][D + 4]
    if (!__syncthreads_and(ptx::mbar_wait(bar_k, 0))) {
        // A late copy may still land in this CTA's shared memory: one more bounded
        // wait for both before the CTA retires.
        ptx::mbar_wait(bar_k, 0);
        ptx::mbar_wait(bar_v, 0);
        if (tid == 0) report(A.status, GQA_DEV_TIMEOUT);
        return;
    }

    const int r = lane >> 2, kk = lane & 3;
    // q as the 8-column operand: column r is head r (WIDE) or r & 3.  Word kk of group
    // g covers coordinates 16 g + 4 kk .. + 3 and their partners in the second half;
    // code_pair(w, 0), (w, 4), (w, 8), (w, 12) are coordinates (0, 2) of the first
    // half, of the second, (1, 3) of the first, of the second.
    uint32_t bq[NG][4];
    float qsum[NG][2];                 // sum of q over the group, heads of columns 2kk, 2kk+1
    {
        const int hr = WIDE ? r : (r & 3);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            uint2 lo = make_uint2(0, 0), hi = make_uint2(0, 0);
            if (hr < G) {
                lo = *reinterpret_cast<const uint2 *>(qs + hr * D + 16 * g + 4 * kk);
                hi = *reinterpret_cast<const uint2 *>(qs + hr * D + D / 2 + 16 * g + 4 * kk);
            }
            bq[g][0] = __byte_perm(lo.x, lo.y, 0x5410);
            bq[g][1] = __byte_perm(hi.x, hi.y, 0x5410);
            bq[g][2] = __byte_perm(lo.x, lo.y, 0x7632);
            bq[g][3] = __byte_perm(hi.x, hi.y, 0x7632);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            constexpr uint32_t one = 0x3f803f80u;
            mma_bf16(acc, one, one, one, one, bq[g][0], bq[g][1]);
            mma_bf16(acc, one, one, one, one, bq[g][2], bq[g][3]);
            qsum[g][0] = acc[0];
            qsum[g][1] = acc[1];
        }
    }

    // ---- scores of the warp's tiles: tile i holds keys 16 (4 i + warp) .. + 15 ----
    // Lane (r, kk) has keys r and r + 8 of the tile against columns 2 kk, 2 kk + 1.
    float sc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t0 = 16 * (kWarps * i + warp);
        sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = -INFINITY;
        if (t0 < nk) {                                     // uniform across the warp
            uint32_t w0[NG], w1[NG], m0[NG], m1[NG];
            load_words<NG>(w0, kw + (t0 + r) * S::kRowWords + NG * kk);
            load_words<NG>(w1, kw + (t0 + r + 8) * S::kRowWords + NG * kk);
            load_words<NG>(m0, ksw + (t0 + r) * NG);
            load_words<NG>(m1, ksw + (t0 + r + 8) * NG);
            float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                mma_bf16(acc, code_pair(w0[g], 0), code_pair(w1[g], 0), code_pair(w0[g], 4),
                         code_pair(w1[g], 4), bq[g][0], bq[g][1]);
                mma_bf16(acc, code_pair(w0[g], 8), code_pair(w1[g], 8), code_pair(w0[g], 12),
                         code_pair(w1[g], 12), bq[g][2], bq[g][3]);
                const float s0 = bf16lo(m0[g]), s1 = bf16lo(m1[g]);
                const float z0 = fmaf(-128.f, s0, bf16hi(m0[g]));
                const float z1 = fmaf(-128.f, s1, bf16hi(m1[g]));
                ptx::ffma2(a0, a1, s0, s0, acc[0], acc[1], a0, a1);
                ptx::ffma2(a0, a1, z0, z0, qsum[g][0], qsum[g][1], a0, a1);
                ptx::ffma2(a2, a3, s1, s1, acc[2], acc[3], a2, a3);
                ptx::ffma2(a2, a3, z1, z1, qsum[g][0], qsum[g][1], a2, a3);
            }
            if (t0 + r < nk) {
                sc[i][0] = a0 * A.scale_log2;
                sc[i][1] = a1 * A.scale_log2;
            }
            if (t0 + r + 8 < nk) {
                sc[i][2] = a2 * A.scale_log2;
                sc[i][3] = a3 * A.scale_log2;
            }
        }
    }

    // ---- the warp's softmax statistics (base 2) per column ----
    float mw[2], lw[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NT; ++i) m = fmaxf(m, fmaxf(sc[i][e], sc[i][e + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float ref = m == -INFINITY ? 0.f : m;        // a warp with no live key
        float l = 0.f;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            sc[i][e] = ex2(sc[i][e] - ref);
            sc[i][e + 2] = ex2(sc[i][e + 2] - ref);
            l += sc[i][e] + sc[i][e + 2];
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        mw[e] = m;
        lw[e] = l;
    }

    // ---- output: rows = coordinates, columns = heads ----
    if (!__syncthreads_and(ptx::mbar_wait(bar_v, 0))) {
        ptx::mbar_wait(bar_v, 0);
        if (tid == 0) report(A.status, GQA_DEV_TIMEOUT);
        return;
    }
    float o[NG][2][4];                 // [g][jj]: coordinates 16 g + 2 r + jj, D/2 + the same
    float off[NG][4];                  // 128 sum(p s), the same in every row
    float pm[NG][2];                   // this lane's keys' share of sum(p m)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[g][0][e] = o[g][1][e] = off[g][e] = 0.f;
        pm[g][0] = pm[g][1] = 0.f;
    }
    // Columns 4 .. 7 hold what bf16 left of columns 0 .. 3 (not WIDE).
    const uint32_t rest = !WIDE && kk >= 2 ? 0xffffffffu : 0u;
    const uint32_t sel = (r & 1) ? 0x7632u : 0x5410u;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int t0 = 16 * (kWarps * i + warp);
        if (t0 < nk) {                                     // uniform across the warp
            uint32_t m0[NG], m1[NG], wa[NG], wb[NG], wc[NG], wd[NG];
            load_words<NG>(m0, vsw + (t0 + r) * NG);
            load_words<NG>(m1, vsw + (t0 + r + 8) * NG);
            const uint32_t *vr = vw + (t0 + 2 * kk) * S::kRowWords + NG * (r >> 1);
            load_words<NG>(wa, vr);
            load_words<NG>(wb, vr + S::kRowWords);
            load_words<NG>(wc, vr + 8 * S::kRowWords);
            load_words<NG>(wd, vr + 9 * S::kRowWords);
            const bool live0 = t0 + r < nk, live1 = t0 + r + 8 < nk;
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                // Rows behind the length may hold anything: their scales count as 0.
                const uint32_t x0 = live0 ? m0[g] : 0u, x1 = live1 ? m1[g] : 0u;
                const float s0 = bf16lo(x0), s1 = bf16lo(x1);
                ptx::ffma2(pm[g][0], pm[g][1], bf16hi(x0), bf16hi(x0), sc[i][0], sc[i][1],
                           pm[g][0], pm[g][1]);
                ptx::ffma2(pm[g][0], pm[g][1], bf16hi(x1), bf16hi(x1), sc[i][2], sc[i][3],
                           pm[g][0], pm[g][1]);
                const float p0 = sc[i][0] * s0, p1 = sc[i][1] * s0;
                const float p2 = sc[i][2] * s1, p3 = sc[i][3] * s1;
                uint32_t h01 = pack_bf16x2(p0, p1), h23 = pack_bf16x2(p2, p3);
                const uint32_t y0 = __byte_perm(wa[g], wb[g], sel);
                const uint32_t y1 = __byte_perm(wc[g], wd[g], sel);
                const uint32_t c00 = code_pair(y0, 0), c01 = code_pair(y0, 4);
                const uint32_t c02 = code_pair(y1, 0), c03 = code_pair(y1, 4);
                const uint32_t c10 = code_pair(y0, 8), c11 = code_pair(y0, 12);
                const uint32_t c12 = code_pair(y1, 8), c13 = code_pair(y1, 12);
                constexpr uint32_t k128 = 0x43004300u;
                if constexpr (WIDE) {
                    const uint32_t l01 = pack_bf16x2(p0 - bf16lo(h01), p1 - bf16hi(h01));
                    const uint32_t l23 = pack_bf16x2(p2 - bf16lo(h23), p3 - bf16hi(h23));
                    const uint32_t b0 = transpose8(l01), b1 = transpose8(l23);
                    mma_bf16(o[g][0], c00, c01, c02, c03, b0, b1);
                    mma_bf16(o[g][1], c10, c11, c12, c13, b0, b1);
                    mma_bf16(off[g], k128, k128, k128, k128, b0, b1);
                } else {
                    const uint32_t r01 = h01 & rest, r23 = h23 & rest;
                    h01 = pack_bf16x2(p0 - bf16lo(r01), p1 - bf16hi(r01));
                    h23 = pack_bf16x2(p2 - bf16lo(r23), p3 - bf16hi(r23));
                }
                const uint32_t b0 = transpose8(h01), b1 = transpose8(h23);
                mma_bf16(o[g][0], c00, c01, c02, c03, b0, b1);
                mma_bf16(o[g][1], c10, c11, c12, c13, b0, b1);
                mma_bf16(off[g], k128, k128, k128, k128, b0, b1);
            }
        }
    }
    __syncthreads();                   // every warp is done with the codes: partials go there
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        float d0 = pm[g][0], d1 = pm[g][1];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            d0 += __shfl_xor_sync(0xffffffffu, d0, x);
            d1 += __shfl_xor_sync(0xffffffffu, d1, x);
        }
        d0 = (rest ? 0.f : d0) - off[g][0];
        d1 = (rest ? 0.f : d1) - off[g][1];
        float *p0 = part + (warp * kCols + 2 * kk) * S::kPartStride + 16 * g + 2 * r;
        float *p1 = p0 + S::kPartStride;
        *reinterpret_cast<float2 *>(p0) = make_float2(o[g][0][0] + d0, o[g][1][0] + d0);
        *reinterpret_cast<float2 *>(p0 + D / 2) = make_float2(o[g][0][2] + d0, o[g][1][2] + d0);
        *reinterpret_cast<float2 *>(p1) = make_float2(o[g][0][1] + d1, o[g][1][1] + d1);
        *reinterpret_cast<float2 *>(p1 + D / 2) = make_float2(o[g][0][3] + d1, o[g][1][3] + d1);
    }
    if (r == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            wml[(warp * kCols + 2 * kk + e) * 2] = mw[e];
            wml[(warp * kCols + 2 * kk + e) * 2 + 1] = lw[e];
        }
    }
    __syncthreads();

    // ---- merge the warps ----
    const size_t row0 = ((size_t)b * A.Hq + h0) * A.n_splits + c;
    if (tid < G) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wml[(w * kCols + tid) * 2]);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float m = wml[(w * kCols + tid) * 2];
            const float f = m == -INFINITY ? 0.f : ex2(m - M);
            sw[w * kCols + tid] = f;
            L = fmaf(f, wml[(w * kCols + tid) * 2 + 1], L);
        }
        s_inv[tid] = 1.f / L;
        if (A.n_splits > 1) {
            A.ws_ml[(row0 + (size_t)tid * A.n_splits) * 2] = M;
            A.ws_ml[(row0 + (size_t)tid * A.n_splits) * 2 + 1] = L;
        }
    }
    __syncthreads();
    for (int idx = tid; idx < G * (D / 2); idx += kThreads) {
        const int h = idx / (D / 2), d = 2 * (idx - h * (D / 2));
        float a0 = 0.f, a1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = sw[w * kCols + h];
            float2 v = *reinterpret_cast<const float2 *>(part + (w * kCols + h) * S::kPartStride + d);
            if constexpr (!WIDE) {
                const float2 v2 = *reinterpret_cast<const float2 *>(
                    part + (w * kCols + h + 4) * S::kPartStride + d);
                v.x += v2.x;
                v.y += v2.y;
            }
            a0 = fmaf(f, v.x, a0);
            a1 = fmaf(f, v.y, a1);
        }
        if (A.n_splits == 1) {
            const float inv = s_inv[h];
            *reinterpret_cast<uint32_t *>(A.out + ((size_t)b * A.Hq + h0 + h) * D + d) =
                pack_bf16x2(a0 * inv, a1 * inv);
        } else {
            *reinterpret_cast<float2 *>(A.ws_o + (row0 + (size_t)h * A.n_splits) * D + d) =
                make_float2(a0, a1);
        }
    }
}

// Merges the chunks of each (sequence, query head) row.  WPR warps share a row and
// take groups of 32 of its chunks in turn, lane i owning coordinates 4 i .. 4 i + 3:
// all partials of a group are loaded before any is used, lane i holds chunk i's
// (m, l), and the weights travel by shuffle.
template <int D, int WPR>
__global__ void __launch_bounds__(128)
decode_q4_merge_kernel(const float *__restrict__ ws_ml, const float *__restrict__ ws_o,
                       const int32_t *__restrict__ lens, int max_len, int Hq, int Lmax, int chunk,
                       int n_splits, int n_rows, uint16_t *__restrict__ out) {
    __shared__ float sm[4], sl[4];
    __shared__ __align__(16) float so[4][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * (4 / WPR) + warp / WPR;
    const int part = warp % WPR;
    if (WPR == 1 && row >= n_rows) return;                 // WPR == 4: the grid is n_rows
    const int b = row / Hq;
    const int len = lens[b];
    uint16_t *o = out + (size_t)row * D;
    constexpr int kLanes = D / 4;
    const bool live = lane < kLanes;
    if (len < 1 || len > max_len || len > Lmax) {          // uniform over the row's warps
        if (live && part == 0) *reinterpret_cast<uint2 *>(o + lane * 4) = make_uint2(0, 0);
        return;
    }
    const int ns = (len + chunk - 1) / chunk;
    const float *ml = ws_ml + (size_t)row * n_splits * 2;
    const float *po = ws_o + (size_t)row * n_splits * D + lane * 4;
    float M = -INFINITY, L = 0.f;
    float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
    for (int base = 32 * part; base < ns; base += 32 * WPR) {
        const int n = min(32, ns - base);
        float4 pv[32];
#pragma unroll
        for (int jj = 0; jj < 32; ++jj)
            pv[jj] = (live && jj < n)
                         ? *reinterpret_cast<const float4 *>(po + (size_t)(base + jj) * D)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        const float2 mi = lane < n ? *reinterpret_cast<const float2 *>(ml + 2 * (base + lane))
                                   : make_float2(-INFINITY, 0.f);
        const float mn = fmaxf(M, warp_max(mi.x));
        const float alpha = M == -INFINITY ? 0.f : ex2(M - mn);
        const float w = lane < n ? ex2(mi.x - mn) : 0.f;
        L = fmaf(L, alpha, warp_sum(w * mi.y));
        a0 *= alpha;
        a1 *= alpha;
        a2 *= alpha;
        a3 *= alpha;
        M = mn;
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
            const float wj = __shfl_sync(0xffffffffu, w, jj);
            a0 = fmaf(wj, pv[jj].x, a0);
            a1 = fmaf(wj, pv[jj].y, a1);
            a2 = fmaf(wj, pv[jj].z, a2);
            a3 = fmaf(wj, pv[jj].w, a3);
        }
    }
    if constexpr (WPR > 1) {
        if (lane == 0) {
            sm[warp] = M;
            sl[warp] = L;
        }
        if (live) *reinterpret_cast<float4 *>(&so[warp][lane * 4]) = make_float4(a0, a1, a2, a3);
        __syncthreads();
        if (warp != 0) return;
        float top = sm[0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) top = fmaxf(top, sm[w]);
        L = a0 = a1 = a2 = a3 = 0.f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) {
            const float f = sm[w] == -INFINITY ? 0.f : ex2(sm[w] - top);
            L = fmaf(f, sl[w], L);
            if (live) {
                const float4 v = *reinterpret_cast<const float4 *>(&so[w][lane * 4]);
                a0 = fmaf(f, v.x, a0);
                a1 = fmaf(f, v.y, a1);
                a2 = fmaf(f, v.z, a2);
                a3 = fmaf(f, v.w, a3);
            }
        }
    }
    if (live) {
        const float inv = 1.f / L;
        *reinterpret_cast<uint2 *>(o + lane * 4) =
            make_uint2(pack_bf16x2(a0 * inv, a1 * inv), pack_bf16x2(a2 * inv, a3 * inv));
    }
}

// How a call is cut: heads per CTA, tiles per warp, chunks of a sequence.
struct Plan {
    int G, n_sub, nt, n_splits;
};

Plan make_plan(int B, int Hq, int Hkv, int max_len) {
    Plan P;
    const int g = Hq / Hkv;
    P.n_sub = (g + kCols - 1) / kCols;
    P.G = (g + P.n_sub - 1) / P.n_sub;
    P.n_sub = (g + P.G - 1) / P.G;
    const long long rows = (long long)B * Hkv * P.n_sub;
    // Longer chunks leave fewer partials; shorter ones spread a small call over more
    // SMs.  The longest that still gives every SM its four resident CTAs.
    P.nt = 4;
    while (P.nt > 1 && rows * ((max_len + 64 * P.nt - 1) / (64 * P.nt)) < 148 * 4) P.nt >>= 1;
    P.n_splits = (max_len + 64 * P.nt - 1) / (64 * P.nt);
    return P;
}

template <int D, int NT, bool WIDE>
cudaError_t launch_split(const DecQ4Args &A, cudaStream_t s) {
    using S = DecQ4Shape<D, NT>;
    auto kern = decode_q4_kernel<D, NT, WIDE>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(A.n_splits, A.Hkv * A.n_sub, A.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, A);
}

template <int D>
cudaError_t launch_decode(const DecQ4Args &A, int nt, cudaStream_t s) {
    const bool wide = A.G > 4;
    cudaError_t e;
    switch (nt) {
        case 1: e = wide ? launch_split<D, 1, true>(A, s) : launch_split<D, 1, false>(A, s); break;
        case 2: e = wide ? launch_split<D, 2, true>(A, s) : launch_split<D, 2, false>(A, s); break;
        default: e = wide ? launch_split<D, 4, true>(A, s) : launch_split<D, 4, false>(A, s); break;
    }
    if (e != cudaSuccess || A.n_splits == 1) return e;
    const int rows = A.B * A.Hq;
    if (A.n_splits > 32)               // one group of 32 chunks is one warp's work
        return launch_pdl(decode_q4_merge_kernel<D, 4>, (unsigned)rows, 128, s,
                          (const float *)A.ws_ml, (const float *)A.ws_o, A.lens, A.max_len, A.Hq,
                          A.Lmax, 64 * nt, A.n_splits, rows, A.out);
    return launch_pdl(decode_q4_merge_kernel<D, 1>, (unsigned)((rows + 3) / 4), 128, s,
                      (const float *)A.ws_ml, (const float *)A.ws_o, A.lens, A.max_len, A.Hq,
                      A.Lmax, 64 * nt, A.n_splits, rows, A.out);
}

// ---------------------------------------------------------------------------
// reading a 4-bit cache back
// ---------------------------------------------------------------------------
// k_out[b, h, i, :] = bf16(m + s c) of slot first[b] + i, i < count[b]; V likewise.
// Bound by memory (a D = 128 row is 80 bytes in, 256 out).  A warp takes 8 rows of K
// and the same of V at a time: lane 4 r + k holds block k of row r -- word k of every
// group -- and writes, per group and half, four neighbouring values; a row's four
// lanes fill whole 32-byte sectors.
constexpr int kReadRows = 64;          // rows per CTA: two passes of 8 for each warp

struct ReadArgs {
    const uint32_t *codes[2], *scales[2];                  // K, V
    uint16_t *out[2];
    const int32_t *first, *count;
    int32_t *status;
    int Hkv, Lmax, Lout;
};

template <int D>
__global__ void __launch_bounds__(kThreads)
read_q4_kernel(const ReadArgs A) {
    constexpr int NG = Q4Shape<D>::NG;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int h = blockIdx.y, b = blockIdx.z;
    const int f = A.first ? A.first[b] : 0;
    const int n = A.count ? A.count[b] : A.Lout;
    if (f < 0 || n < 0 || n > A.Lout || (long long)f + n > A.Lmax) {
        if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
            report(A.status, f < 0 || n < 0 ? GQA_DEV_BAD_LEN : GQA_DEV_CAPACITY);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane >> 2, kk = lane & 3;
    const int i0 = blockIdx.x * kReadRows + 8 * warp + r;
    uint32_t w[2][2][NG], sm[2][2][NG];                    // [pass][K, V]
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = i0 + 32 * u;
        if (i < n) {
            const size_t row = ((size_t)b * A.Hkv + h) * A.Lmax + f + i;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                load_words<NG>(w[u][t], A.codes[t] + row * (D / 8) + NG * kk);
                load_words<NG>(sm[u][t], A.scales[t] + row * NG);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = i0 + 32 * u;
        if (i < n) {
            const size_t row = ((size_t)b * A.Hkv + h) * A.Lout + i;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint16_t *dst = A.out[t] + row * D + 4 * kk;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float s = bf16lo(sm[u][t][g]), m = bf16hi(sm[u][t][g]);
                    float v[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)            // code + 2^23, then the 2^23 away
                        v[e] = __uint_as_float(((w[u][t][g] >> (4 * e)) & 15u) | 0x4b000000u) -
                               8388608.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = fmaf(s, v[e], m);
                    *reinterpret_cast<uint2 *>(dst + 16 * g) =
                        make_uint2(pack_bf16x2(v[0], v[2]), pack_bf16x2(v[4], v[6]));
                    *reinterpret_cast<uint2 *>(dst + D / 2 + 16 * g) =
                        make_uint2(pack_bf16x2(v[1], v[3]), pack_bf16x2(v[5], v[7]));
                }
            }
        }
    }
}

template <int D>
cudaError_t launch_read(const ReadArgs &A, int B, cudaStream_t s) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((A.Lout + kReadRows - 1) / kReadRows), A.Hkv, B);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, read_q4_kernel<D>, A);
}

}  // namespace
}  // namespace gqa

extern "C" gqa_status kv_cache_read_q4(const void *k_codes, const void *k_scales,
                                       const void *v_codes, const void *v_scales,
                                       const int32_t *first, const int32_t *count, void *k_out,
                                       void *v_out, int B, int Hkv, int D, int Lmax, int Lout,
                                       int32_t *status_dev, void *stream) {
    using namespace gqa_host;
    if (!k_codes || !k_scales || !v_codes || !v_scales || !k_out || !v_out || B < 1 || Hkv < 1 ||
        Lmax < 1 || Lout < 1 || B > 65535 || Hkv > 65535)
        return GQA_ERR_INVALID_ARG;
    if (!aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) ||
        !aligned16(v_scales) || !aligned16(k_out) || !aligned16(v_out) ||
        (reinterpret_cast<uintptr_t>(first) & 3u) || (reinterpret_cast<uintptr_t>(count) & 3u))
        return GQA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return GQA_ERR_UNSUPPORTED;
    if (Lmax % 128 != 0) return GQA_ERR_INVALID_ARG;
    if (!count && Lout > Lmax) return GQA_ERR_CAPACITY;
    gqa::ReadArgs A = {};
    A.codes[0] = static_cast<const uint32_t *>(k_codes);
    A.codes[1] = static_cast<const uint32_t *>(v_codes);
    A.scales[0] = static_cast<const uint32_t *>(k_scales);
    A.scales[1] = static_cast<const uint32_t *>(v_scales);
    A.out[0] = static_cast<uint16_t *>(k_out);
    A.out[1] = static_cast<uint16_t *>(v_out);
    A.first = first;
    A.count = count;
    A.status = status_dev;
    A.Hkv = Hkv;
    A.Lmax = Lmax;
    A.Lout = Lout;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 64   ? gqa::launch_read<64>(A, B, s)
                          : D == 96 ? gqa::launch_read<96>(A, B, s)
                                    : gqa::launch_read<128>(A, B, s);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

extern "C" size_t gqa_decode_q4_workspace_bytes(int B, int Hq, int Hkv, int D, int max_len) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_len < 1 || !gqa_host::head_dim_ok(D))
        return 0;
    const gqa::Plan P = gqa::make_plan(B, Hq, Hkv, max_len);
    if (P.n_splits == 1) return 16;                        // the chunk's CTA writes the output
    const size_t rows = (size_t)B * Hq * P.n_splits;
    // The partial outputs start on a 16-byte boundary.
    return (rows * 2 * 4 + 15) / 16 * 16 + rows * (size_t)D * 4;
}

extern "C" gqa_status gqa_decode_q4(const void *q, const void *k_codes, const void *k_scales,
                                    const void *v_codes, const void *v_scales,
                                    const int32_t *lens, int max_len_host, void *out, int B,
                                    int Hq, int Hkv, int D, int Lmax, float scale, void *ws,
                                    size_t ws_bytes, int32_t *status_dev, void *stream) {
    using namespace gqa_host;
    if (!q || !k_codes || !k_scales || !v_codes || !v_scales || !lens || !out || B < 1 || Hq < 1 ||
        Hkv < 1 || Lmax < 1)
        return GQA_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || B > 65535 || Hq > 65535) return GQA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) ||
        !aligned16(v_scales) || !aligned16(out) || (reinterpret_cast<uintptr_t>(lens) & 3u))
        return GQA_ERR_INVALID_ARG;
    if (!head_dim_ok(D)) return GQA_ERR_UNSUPPORTED;
    if (Lmax % 128 != 0) return GQA_ERR_INVALID_ARG;
    if (max_len_host < 1) return GQA_ERR_INVALID_ARG;
    if (max_len_host > Lmax) return GQA_ERR_CAPACITY;
    const size_t need = gqa_decode_q4_workspace_bytes(B, Hq, Hkv, D, max_len_host);
    const gqa::Plan P = gqa::make_plan(B, Hq, Hkv, max_len_host);
    if (P.n_splits > 1 && (!ws || ws_bytes < need || !aligned16(ws))) return GQA_ERR_WORKSPACE;
    gqa::DecQ4Args A = {};
    A.q = static_cast<const uint16_t *>(q);
    A.kc = static_cast<const uint8_t *>(k_codes);
    A.ks = static_cast<const uint32_t *>(k_scales);
    A.vc = static_cast<const uint8_t *>(v_codes);
    A.vs = static_cast<const uint32_t *>(v_scales);
    A.lens = lens;
    A.out = static_cast<uint16_t *>(out);
    A.ws_ml = static_cast<float *>(ws);
    const size_t rows = (size_t)B * Hq * P.n_splits;
    A.ws_o = A.ws_ml + (rows * 2 + 3) / 4 * 4;
    A.status = status_dev;
    A.max_len = max_len_host;
    A.B = B;
    A.Hq = Hq;
    A.Hkv = Hkv;
    A.Lmax = Lmax;
    A.n_splits = P.n_splits;
    A.n_sub = P.n_sub;
    A.G = P.G;
    A.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 64   ? gqa::launch_decode<64>(A, P.nt, s)
                          : D == 96 ? gqa::launch_decode<96>(A, P.nt, s)
                                    : gqa::launch_decode<128>(A, P.nt, s);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}
