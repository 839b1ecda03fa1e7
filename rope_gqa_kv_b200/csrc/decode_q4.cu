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
//   * a 4-bit number in the low bits of a 16-bit float is a subnormal: c stands for
//     c 2^-133 in bf16 and c 2^-24 in fp16, and four bits higher for 16 times that,
//     all exact in the product.  One AND of a word of codes so gives two of them
//     (code_pair); a word's eight codes take five instructions.  Codes are the
//     16-row operand of mma.m16n8k16 (rows = keys for the scores, coordinates for the
//     output) and the query heads its 8 columns: a group of heads costs what one
//     head costs.
//   * scores: q stays bf16, times 2^64 (2^60 against the codes four bits up), so the
//     products are exact; a key's s multiplies the sum of its group.  The minima's
//     part, sum over groups of m sum(q), is one more product whose 16-row operand is
//     the (s, m) words themselves, with sum(q) in three bf16 parts (24 bits).
//   * output: sum_k p_k (m_k + s_k c_k,d).  p_k s_k is the 8-column operand, carried
//     by movmatrix from the score layout, in fp16 after a power of two that brings the
//     group's largest s so far to 2^5 .. 2^6: one rounding, 2^-11 of the term, against
//     bf16's 2^-8 (terms below 2^-19 of the group's largest lose bits, 2^-30 of it at
//     most).
//     sum(p m) is added up in fp32 beside it.
//   * the codes are never negative and the minima take most of their sum away again, while
//     the tensor cores cut every product off at the last place of the sum so far: over
//     a long chunk a loss of some 2^-23 of that sum for every 16 keys, all one way.  Every
//     kCentre units the sums are therefore moved past zero by what one coordinate has
//     gathered, and that amount goes over to sum(p m): neither changes the result, and the
//     loss no longer grows with the chunk.
// mma.sync rather than tcgen05: its operands come from registers, where the codes
// are unpacked; tcgen05 would need them written to shared memory as bf16, four
// times the bytes that arrived, for 8 columns of work.
//
// Work: one CTA per (chunk of the cached slots, KV head x head subgroup, sequence); with
// few rows the chunks are shared out by the lengths on the device (even_chunk).
// Its four warps take the chunk's units of kTiles 16-key tiles in turn, each through a ring
// of its own (asynchronous 16-byte copies; no warp waits for another), with a
// running softmax: the reference moves, and what is summed is scaled down, only when a
// score passes it by more than 8, i.e. hardly ever after the first tile.  References and
// the chunks' m are scores before scaling: the largest is then exactly 0 from itself, while
// against a rounded product it would be off by 2^-24 of the score, more than an exponent's
// range for scores from 2^31 on.  At the end
// the warps' statistics and partial outputs are merged in shared memory, the chunk's
// (m, l, o) goes to the workspace and a second kernel, a programmatic dependent,
// merges the chunks.  When one chunk covers max_len the CTA writes the output itself.
// Calls of few, short rows (make_plan) merge without a second kernel: a row's CTAs are a
// thread-block cluster, each hands its (m, l, o) to the first one's shared memory, and
// that one writes the output.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "q4.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace gqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kResident = 3;           // CTAs per SM
constexpr int kTiles = 2;              // tiles of 16 keys that a warp takes at a time
constexpr int kStages = 3;             // such units in a warp's ring
constexpr int kCols = 8;               // columns of the mma: query heads of a CTA, at most
constexpr int kMaxCluster = 8;         // CTAs of a cluster
// Units between two moves of the sums past zero.  The error for 10^6 normal keys of 24 / 8
// heads, D = 128, is 0.0224 of the output without, 0.0018 with 16 or 8 (0.0017 is the output's
// rounding to bf16); 4 x 57000 keys 0.0020 and 0.0017.  8 x 32768 slots take 67.5 us without,
// 68.5 with 16, 69.7 with 8; 256 x 256 .. 2048 85.1, 86.3 and 87.3.
constexpr int kCentre = 16;
constexpr float kSlack = 8.0f;         // a score may pass the softmax reference by this (log2)
constexpr float kNoRef = -3.402823466e38f;   // before any score: the lowest finite value, so that
                                       // 2^(a score of -inf - it) is 0

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with 8 columns of the first operand.
__device__ __forceinline__ void mma_bf16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
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

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two codes of a word as subnormal numbers: those in the low four bits of each half,
// and the ones above them (16 times as large).
__device__ __forceinline__ uint32_t code_pair(uint32_t w) { return w & 0x000f000fu; }
__device__ __forceinline__ uint32_t code_pair16(uint32_t w) { return w & 0x00f000f0u; }

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

// Cluster: the barrier, and stores to the first CTA's shared memory.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_first_cta(uint32_t smem) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem));
    return a;
}
__device__ __forceinline__ void store_remote(uint32_t at, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(x), "f"(y) : "memory");
}

template <int D>
struct DecQ4Shape {
    static constexpr int NG = Q4Shape<D>::NG;
    static constexpr int RB = D / 2;                       // bytes of codes per row
    static constexpr int SB = 4 * NG;                      // bytes of scales per row
    static constexpr int R = 16 * kTiles;                  // rows of a unit
    // Bytes from row to row in the ring.  D = 128: 80, so that neither the two rows
    // that eight lanes read of K nor the four they read of V meet in a bank.
    static constexpr int RS = D == 128 ? 80 : RB;
    // A unit in the ring: [K codes][V codes][K scales][V scales].
    static constexpr int kOffV = R * RS;
    static constexpr int kOffKS = 2 * R * RS;
    static constexpr int kOffVS = 2 * R * RS + R * SB;
    static constexpr int kUnit = 2 * R * (RS + SB);
    static constexpr int kRing = kWarps * kStages * kUnit;
    // The warps' partial outputs (kWarps x kCols x (D + 4) f32) are written over the
    // rings once every warp is done.  D + 4: the four lanes of a row write four
    // columns, 8 banks apart.
    static constexpr int kPartStride = D + 4;
    static constexpr int kPart = kWarps * kCols * kPartStride * 4;
    static constexpr int kSmem = kRing > kPart ? kRing : kPart;
    // Clusters: what each CTA hands to the first one, over its ring: o [kCols][D],
    // (m, l) [kCols].
    static constexpr int kGather = kCols * (D + 2) * 4;
    static_assert(kMaxCluster * kGather <= kSmem, "the parts of a cluster fit over a ring");
};

struct DecQ4Args {
    const uint16_t *q;
    const uint8_t *kc, *vc;
    const uint32_t *ks, *vs;
    const int32_t *lens;
    uint16_t *out;
    float *ws_ml, *ws_o;
    int32_t *status;
    int max_len, B, Hq, Hkv, Lmax, n_sub, G;               // G: query heads per CTA
    int chunk, n_splits;                                   // slots per CTA, chunks of max_len
    int places;                                            // or: chunks to share out, see even_chunk
    int cluster;                                           // CTAs of a row's cluster, or 0
    float scale_log2;                  // 2^69 scale / ln 2: the scores come in units of 2^-69
    float slack;                       // kSlack in the scores' units
};

// Calls of few rows share `places` chunks among their sequences by the lengths that these
// have: the shortest chunk, a multiple of 64 slots, of which the sequences (lane b holds
// sequence b's length; one that is out of range and lanes without one hold 0) take no more
// than that, one each at least.  With S slots in all, sum of ceil(len / c) <= S / c + B, so
// c = S / (places - B) does, and c < S / places does not.
__device__ __forceinline__ int chunks_of(int len, int chunk, bool mine) {
    return mine ? max(1, (len + chunk - 1) / chunk) : 0;
}
__device__ __forceinline__ int even_chunk(int len, bool mine, int B, int places) {
    const int S = __reduce_add_sync(0xffffffffu, len);     // B max_len < 2^30
    int lo = max(1, (S / places + 63) / 64);               // in 64 slots
    int hi = max(lo, S / (places - B) / 64 + 1);
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__reduce_add_sync(0xffffffffu, chunks_of(len, 64 * mid, mine)) <= places) hi = mid;
        else lo = mid + 1;
    }
    return 64 * lo;
}
// Sequence b's length, 0 where it is out of range.
__device__ __forceinline__ int len_or_zero(const int32_t *lens, int b, int max_len, int Lmax) {
    const int len = lens[b];
    return len < 1 || len > max_len || len > Lmax ? 0 : len;
}

// Workspace: [(m, l): rows x 2 f32][o: rows x D f32], rows = B x Hq x n_splits, row
// (b, h, c) = (b * Hq + h) * n_splits + c.
template <int D, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, kResident)
decode_q4_kernel(const DecQ4Args A) {
    using S = DecQ4Shape<D>;
    constexpr int NG = S::NG, U = kTiles;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float wml[kWarps * kCols * 2];              // (m, l) [warp][column]
    __shared__ float sw[kWarps * kCols];                   // merge weights [warp][column]
    __shared__ float s_inv[kCols];

    // Wait for the kernel before this one (normally the append that wrote lens and
    // the newest slot) before reading; the merge may then be scheduled.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // Chunks in the slowest order: those behind the shorter sequences' ends, which have
    // nothing to do, come last.
    int c = blockIdx.z, b = blockIdx.y, chunk = A.chunk;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!CLUSTER && A.places) {                            // b and c from the lengths
        const bool mine = lane < A.B;
        const int mylen = mine ? len_or_zero(A.lens, lane, A.max_len, A.Lmax) : 0;
        chunk = even_chunk(mylen, mine, A.B, A.places);
        const int n = chunks_of(mylen, chunk, mine);
        int end = n;                                       // the first chunk behind the lane's
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, end, x);
            if (lane >= x) end += y;
        }
        b = __popc(__ballot_sync(0xffffffffu, end <= c));
        if (b >= A.B) return;
        c -= __shfl_sync(0xffffffffu, end - n, b);
    }
    const int kvh = blockIdx.x / A.n_sub, sub = blockIdx.x - kvh * A.n_sub;
    const int group = A.Hq / A.Hkv;
    const int h0 = kvh * group + sub * A.G;                // first query head
    const int G = min(A.G, group - sub * A.G);             // query heads of this CTA
    const int len = A.lens[b];
    if (len < 1 || len > A.max_len || len > A.Lmax) {
        if (c == 0 && blockIdx.x == 0 && tid == 0)
            report(A.status, len < 1 ? GQA_DEV_BAD_LEN : GQA_DEV_CAPACITY);
        if (A.n_splits == 1 || (CLUSTER && c == 0))
            for (int i = tid; i < G * D; i += kThreads) A.out[((size_t)b * A.Hq + h0) * D + i] = 0;
        return;
    }
    const int key0 = c * chunk;
    if (key0 >= len) {
        if constexpr (CLUSTER) {                           // (len is the whole cluster's)
            cluster_arrive();
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    const int nk = min(chunk, len - key0);

    // ---- the warp's ring ----
    // A lane copies 16 bytes of each 512-byte block of codes, and 16 of each 256 of the
    // scales: lanes 0 .. 15 K's, lanes 16 .. 31 V's.
    const size_t row = ((size_t)b * A.Hkv + kvh) * A.Lmax + key0 + warp * S::R;
    const uint8_t *kg = A.kc + row * S::RB + 16 * lane, *vg = A.vc + row * S::RB + 16 * lane;
    const uint8_t *sg = reinterpret_cast<const uint8_t *>(lane < 16 ? A.ks : A.vs) +
                        row * S::SB + 16 * (lane & 15);
    const uint32_t ring = ptx::smem_addr(smem) + warp * (kStages * S::kUnit);
    const int n_units = (nk + S::R - 1) / S::R;
    // Unit u, the warp's next, to a stage.  The rows behind the length are not read: their
    // codes and scales are zeros.
    auto copy = [&](uint32_t dst, int live, auto full) {   // full: no row is behind the length
#pragma unroll
        for (int x = 0; x < S::R * S::RB; x += 512) {
            const int at = x + 16 * lane;                  // in the unit's codes
            if (x + 512 <= S::R * S::RB || at < S::R * S::RB) {
                const uint32_t to = dst + at / S::RB * S::RS + at % S::RB;
                const int n = full ? 16 : min(16, max(0, live * S::RB - at));
                copy16(to, kg + x, n);
                copy16(to + S::kOffV, vg + x, n);
            }
        }
#pragma unroll
        for (int x = 0; x < S::R * S::SB; x += 256) {
            const int at = x + 16 * (lane & 15);
            if (x + 256 <= S::R * S::SB || at < S::R * S::SB)
                copy16(dst + (lane < 16 ? S::kOffKS : S::kOffVS) + at, sg + x,
                       full ? 16 : min(16, max(0, live * S::SB - at)));
        }
    };
    auto fetch = [&](int u, int stage) {
        const int live = nk - S::R * u;                    // uniform across the warp
        if (live >= S::R)
            copy(ring + stage * S::kUnit, live, std::true_type{});
        else
            copy(ring + stage * S::kUnit, live, std::false_type{});
        kg += S::R * kWarps * S::RB;
        vg += S::R * kWarps * S::RB;
        sg += S::R * kWarps * S::SB;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        if (warp + kWarps * i < n_units) fetch(warp + kWarps * i, i);
        copy_commit();
    }

    const int r = lane >> 2, kk = lane & 3;
    // Row r of a product's first eight is key sr of the tile, row r + 8 key sr + 8: any
    // order serves.  With these, what the lanes of one access read lies in different
    // banks: rows (i, i + 4) of K together, or (D = 64) any four neighbours in r, and
    // the rows va (and vb) of V for kk = 0 .. 3.
    const int sr = D == 64 ? ((r >> 1) & 1) + 2 * ((r & 1) ^ (r >> 2)) + (r & 4)
                           : (r >> 1) + 4 * (r & 1);
    const int va = D == 64 ? (kk & 1) + 6 * (kk >> 1) : kk;          // sr of r = 2 kk
    const int vb = D == 64 ? kk + 2 : kk + 4;                        // sr of r = 2 kk + 1
    // q as the 8-column operand: column r is head r.  Word kk of group g covers
    // coordinates 16 g + 4 kk .. + 3 and their partners in the second half; its codes
    // come as coordinates (0, 2) of the first half, of the second (times 16), and,
    // shifted down by 8, (1, 3) of the first, of the second (times 16).
    uint4 bqr[NG];
    uint32_t bm[3];                    // sum of q over group kk, head r: bf16 parts, high half
    {
        const uint16_t *q = A.q + ((size_t)b * A.Hq + h0 + r) * D + 4 * kk;
        uint2 lo[NG], hi[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            lo[g] = hi[g] = make_uint2(0, 0);
            if (r < G) {
                lo[g] = *reinterpret_cast<const uint2 *>(q + 16 * g);
                hi[g] = *reinterpret_cast<const uint2 *>(q + D / 2 + 16 * g);
            }
        }
        float qsum[8];                 // [2 g + e]: heads of columns 2 kk + e
#pragma unroll
        for (int i = 0; i < 8; ++i) qsum[i] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const uint32_t b0 = __byte_perm(lo[g].x, lo[g].y, 0x5410);
            const uint32_t b1 = __byte_perm(hi[g].x, hi[g].y, 0x5410);
            const uint32_t b2 = __byte_perm(lo[g].x, lo[g].y, 0x7632);
            const uint32_t b3 = __byte_perm(hi[g].x, hi[g].y, 0x7632);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            constexpr uint32_t one = 0x3f803f80u;
            mma_bf16(acc, one, one, one, one, b0, b1);
            mma_bf16(acc, one, one, one, one, b2, b3);
            qsum[2 * g] = acc[0];
            qsum[2 * g + 1] = acc[1];
            constexpr uint32_t up64 = 0x5f805f80u, up60 = 0x5d805d80u;   // 2^64, 2^60 twice
            bqr[g] = make_uint4(mul_bf16x2(b0, up64), mul_bf16x2(b1, up60),
                                         mul_bf16x2(b2, up64), mul_bf16x2(b3, up60));
        }
        // Every row r of the sums is alike: lane (r, k) offers group r / 2 of head
        // 2 k + r % 2, and fetches group kk of head r.
        float mine = qsum[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) mine = r == i ? qsum[i] : mine;
        float x = __shfl_sync(0xffffffffu, mine, 4 * (2 * kk + (r & 1)) + (r >> 1));
        x *= 0x1p-69f;                 // the scores' unit: 2^64 2^-133
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            bm[i] = pack_bf16x2(0.f, x);
            x -= bf16hi(bm[i]);
        }
    }

    // State of the running softmax.  Lane (r, kk): columns 2 kk, 2 kk + 1; the sums of
    // p and p m are over the lane's own rows, o over all of them.
    float ref[2] = {kNoRef, kNoRef}, l[2] = {0.f, 0.f};
    float o[NG][2][4];                 // [g][jj]: coordinates 16 g + 2 r + jj, D/2 + the same
    float pm[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[g][0][e] = o[g][1][e] = 0.f;
        pm[g][0] = pm[g][1] = 0.f;
    }
    // p s goes into fp16 times up = 2^(132 - eb), eb the biased exponent of the largest V
    // step of the group so far: p <= 2^kSlack keeps it below 2^15, and steps may grow
    // fourfold before the sums have to follow (cap).  o is in units of 2^(eb - 108), with
    // the codes' 2^-24.  Lane (r, kk) keeps group kk's eb and cap.
    const int gk = min(kk, NG - 1);
    uint32_t eb = 0;
    float cap = 0.f, up[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) up[g] = 0.f;
    const uint32_t sel = (r & 1) ? 0x7632u : 0x5410u;

    int stage = 0;
#pragma unroll 1
    for (int u = warp; u < n_units; u += kWarps) {
        copy_wait<kStages - 2>();
        __syncwarp();
        {
            const int ahead = u + kWarps * (kStages - 1);  // into the stage read last
            if (ahead < n_units) fetch(ahead, stage == 0 ? kStages - 1 : stage - 1);
            copy_commit();
        }
        const uint8_t *unit = smem + (warp * kStages + stage) * S::kUnit;
        stage = stage == kStages - 1 ? 0 : stage + 1;
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(unit);
        const uint32_t *vw = reinterpret_cast<const uint32_t *>(unit + S::kOffV);
        const uint32_t *ksw = reinterpret_cast<const uint32_t *>(unit + S::kOffKS);
        const uint32_t *vsw = reinterpret_cast<const uint32_t *>(unit + S::kOffVS);

        // ---- scores: lane (r, kk) has rows r and r + 8 of a tile against its columns ----
        float sc[U][4];
        uint32_t m0[U][NG], m1[U][NG];                     // V's (s, m)
        uint32_t smax = 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int k0 = 16 * j + sr, k1 = k0 + 8;
            uint32_t w0[NG], w1[NG], x0[NG], x1[NG];
            load_words<NG>(w0, kw + k0 * (S::RS / 4) + NG * kk);
            load_words<NG>(w1, kw + k1 * (S::RS / 4) + NG * kk);
            load_words<NG>(x0, ksw + k0 * NG);
            load_words<NG>(x1, ksw + k1 * NG);
            const uint32_t mk0 = ksw[k0 * NG + gk];
            const uint32_t mk1 = ksw[k1 * NG + gk];
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
#pragma unroll
            for (int x = 0; x < 3; ++x) mma_bf16_k8(sc[j], mk0, mk1, bm[x]);
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                const uint32_t u0 = w0[g] >> 8, u1 = w1[g] >> 8;
                mma_bf16(acc, code_pair(w0[g]), code_pair(w1[g]), code_pair16(w0[g]),
                         code_pair16(w1[g]), bqr[g].x, bqr[g].y);
                mma_bf16(acc, code_pair(u0), code_pair(u1), code_pair16(u0), code_pair16(u1),
                         bqr[g].z, bqr[g].w);
                const float s0 = bf16lo(x0[g]), s1 = bf16lo(x1[g]);
                sc[j][0] = fmaf(s0, acc[0], sc[j][0]);
                sc[j][1] = fmaf(s0, acc[1], sc[j][1]);
                sc[j][2] = fmaf(s1, acc[2], sc[j][2]);
                sc[j][3] = fmaf(s1, acc[3], sc[j][3]);
            }
            load_words<NG>(m0[j], vsw + k0 * NG);
            load_words<NG>(m1[j], vsw + k1 * NG);
            smax = max_bf16x2(smax, max_bf16x2(vsw[k0 * NG + gk],
                                               vsw[k1 * NG + gk]));
        }
        if (S::R * (u + 1) > nk) {                         // the sequence ends in this unit
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (S::R * u + 16 * j + sr >= nk) sc[j][0] = sc[j][1] = -INFINITY;
                if (S::R * u + 16 * j + sr + 8 >= nk) sc[j][2] = sc[j][3] = -INFINITY;
            }
        }

        // ---- the references, where they have to move ----
        float n0 = fmaxf(sc[0][0], sc[0][2]), n1 = fmaxf(sc[0][1], sc[0][3]);
#pragma unroll
        for (int j = 1; j < U; ++j) {
            n0 = fmaxf(n0, fmaxf(sc[j][0], sc[j][2]));
            n1 = fmaxf(n1, fmaxf(sc[j][1], sc[j][3]));
        }
        const bool past = u >= kWarps * kCentre && u / kWarps % kCentre == 0;     // uniform
        if (__any_sync(0xffffffffu, fmaxf(n0 - ref[0], n1 - ref[1]) > A.slack ||
                                        bf16lo(smax) >= cap || past)) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
                smax = max_bf16x2(smax, __shfl_xor_sync(0xffffffffu, smax, x));
            }
            n0 = fmaxf(n0, ref[0]);
            n1 = fmaxf(n1, ref[1]);
            const uint32_t neb = max(eb, min(max((smax >> 7) & 0xffu, 17u), 235u));
            // 2^(eb - neb), 0 at the first unit (where all sums are zero) and below 2^-126
            const float es = neb - eb > 126u ? 0.f : __uint_as_float((127u - (neb - eb)) << 23);
            const float f0 = ex2((ref[0] - n0) * A.scale_log2);
            const float f1 = ex2((ref[1] - n1) * A.scale_log2);
            l[0] *= f0;
            l[1] *= f1;
            eb = neb;
            cap = __uint_as_float((eb + 2u) << 23);                  // 4 times the step's power
            const float mine = __uint_as_float((259u - eb) << 23);   // 2^(132 - eb)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                pm[g][0] *= f0;
                pm[g][1] *= f1;
                up[g] = __shfl_sync(0xffffffffu, mine, g);
                const float fg = __shfl_sync(0xffffffffu, es, g);
                const float h0g = f0 * fg, h1g = f1 * fg;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[g][e][0] *= h0g;
                    o[g][e][1] *= h1g;
                    o[g][e][2] *= h0g;
                    o[g][e][3] *= h1g;
                }
            }
            ref[0] = n0;
            ref[1] = n1;
            // The sums past zero: x is what the first coordinate of the group has gathered,
            // times 1.5 at the first move (from X to -X/2) and 2 at the later ones (from
            // X/2 to -X/2).  Rows r + 8 of the products hold 16 times the upper codes plus
            // the lower ones: 17 x.
            if (past) {
                const float by = u == kWarps * kCentre + warp ? 1.5f : 2.0f;
                const float unit = __uint_as_float((eb + 19u) << 23);    // 2^(eb - 108)
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const float x0 = __shfl_sync(0xffffffffu, o[g][0][0], kk) * by;
                    const float x1 = __shfl_sync(0xffffffffu, o[g][0][1], kk) * by;
                    float down = __shfl_sync(0xffffffffu, unit, g);
                    if (r != 0) down = 0.f;                // pm is added up over r
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        o[g][e][0] -= x0;
                        o[g][e][1] -= x1;
                        o[g][e][2] = fmaf(-17.f, x0, o[g][e][2]);
                        o[g][e][3] = fmaf(-17.f, x1, o[g][e][3]);
                    }
                    pm[g][0] = fmaf(x0, down, pm[g][0]);
                    pm[g][1] = fmaf(x1, down, pm[g][1]);
                }
            }
        }

        // ---- output: rows = coordinates, columns = heads ----
#pragma unroll
        for (int j = 0; j < U; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[j][e] = ex2((sc[j][e] - ref[e & 1]) * A.scale_log2);
            l[0] += sc[j][0] + sc[j][2];
            l[1] += sc[j][1] + sc[j][3];
            uint32_t wa[NG], wb[NG], wc[NG], wd[NG];       // rows 2 kk, 2 kk + 1, and 8 on
            const uint32_t *vr = vw + 16 * j * (S::RS / 4) + NG * (r >> 1);
            load_words<NG>(wa, vr + va * (S::RS / 4));
            load_words<NG>(wb, vr + vb * (S::RS / 4));
            load_words<NG>(wc, vr + (va + 8) * (S::RS / 4));
            load_words<NG>(wd, vr + (vb + 8) * (S::RS / 4));
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const float s0 = bf16lo(m0[j][g]) * up[g], s1 = bf16lo(m1[j][g]) * up[g];
                const float z0 = bf16hi(m0[j][g]), z1 = bf16hi(m1[j][g]);
                pm[g][0] = fmaf(z0, sc[j][0], fmaf(z1, sc[j][2], pm[g][0]));
                pm[g][1] = fmaf(z0, sc[j][1], fmaf(z1, sc[j][3], pm[g][1]));
                const uint32_t b0 = transpose8(pack_f16x2(sc[j][0] * s0, sc[j][1] * s0));
                const uint32_t b1 = transpose8(pack_f16x2(sc[j][2] * s1, sc[j][3] * s1));
                // Rows r + 8 get the whole bytes, 16 times the upper code plus the lower:
                // one instruction fewer, and the lower ones' sums are in rows r.
                const uint32_t y0 = __byte_perm(wa[g], wb[g], sel);
                const uint32_t y1 = __byte_perm(wc[g], wd[g], sel);
                const uint32_t u0 = __byte_perm(y0, 0u, 0x4341), u1 = __byte_perm(y1, 0u, 0x4341);
                mma_f16(o[g][0], code_pair(y0), y0 & 0x00ff00ffu, code_pair(y1), y1 & 0x00ff00ffu,
                        b0, b1);
                mma_f16(o[g][1], code_pair(u0), u0, code_pair(u1), u1, b0, b1);
            }
        }
    }

    // ---- the warp's partials, over the rings ----
    copy_wait<0>();
    __syncthreads();
    float *part = reinterpret_cast<float *>(smem);         // [warp][column][D + 4]
    const float mine = __uint_as_float((eb + 19u) << 23);            // 2^(eb - 108)
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], x);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], x);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const float down = __shfl_sync(0xffffffffu, mine, g), down16 = down * 0.0625f;
        float d0 = pm[g][0], d1 = pm[g][1];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            d0 += __shfl_xor_sync(0xffffffffu, d0, x);
            d1 += __shfl_xor_sync(0xffffffffu, d1, x);
        }
        float *p0 = part + (warp * kCols + 2 * kk) * S::kPartStride + 16 * g + 2 * r;
        float *p1 = p0 + S::kPartStride;
        if (2 * kk < G) {
            *reinterpret_cast<float2 *>(p0) =
                make_float2(fmaf(o[g][0][0], down, d0), fmaf(o[g][1][0], down, d0));
            *reinterpret_cast<float2 *>(p0 + D / 2) =
                make_float2(fmaf(o[g][0][2] - o[g][0][0], down16, d0),
                            fmaf(o[g][1][2] - o[g][1][0], down16, d0));
        }
        if (2 * kk + 1 < G) {
            *reinterpret_cast<float2 *>(p1) =
                make_float2(fmaf(o[g][0][1], down, d1), fmaf(o[g][1][1], down, d1));
            *reinterpret_cast<float2 *>(p1 + D / 2) =
                make_float2(fmaf(o[g][0][3] - o[g][0][1], down16, d1),
                            fmaf(o[g][1][3] - o[g][1][1], down16, d1));
        }
    }
    if (r == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            wml[(warp * kCols + 2 * kk + e) * 2] = ref[e];
            wml[(warp * kCols + 2 * kk + e) * 2 + 1] = l[e];
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
            const float f = ex2((m - M) * A.scale_log2);   // 0 for a warp without a tile
            sw[w * kCols + tid] = f;
            L = fmaf(f, wml[(w * kCols + tid) * 2 + 1], L);
        }
        s_inv[tid] = 1.f / L;
        if constexpr (CLUSTER) {
            wml[2 * tid] = M;
            wml[2 * tid + 1] = L;
        } else if (A.n_splits > 1) {
            A.ws_ml[(row0 + (size_t)tid * A.n_splits) * 2] = M;
            A.ws_ml[(row0 + (size_t)tid * A.n_splits) * 2 + 1] = L;
        }
    }
    __syncthreads();
    constexpr int kPer = kCols * (D / 2) / kThreads;       // pairs of coordinates per thread
    float2 sum[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int idx = tid + i * kThreads;
        const int h = idx / (D / 2), d = 2 * (idx - h * (D / 2));
        sum[i] = make_float2(0.f, 0.f);
        if (h < G) {
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sw[w * kCols + h];
                const float2 v =
                    *reinterpret_cast<const float2 *>(part + (w * kCols + h) * S::kPartStride + d);
                sum[i].x = fmaf(f, v.x, sum[i].x);
                sum[i].y = fmaf(f, v.y, sum[i].y);
            }
        }
    }
    uint32_t hand = 0;                                     // this CTA's place in the first one
    if constexpr (CLUSTER) {
        cluster_arrive();                                  // no CTA needs its ring any more
        cluster_wait();
        hand = in_first_cta(ptx::smem_addr(smem) + c * S::kGather);
        if (tid < G) store_remote(hand + kCols * D * 4 + 8 * tid, wml[2 * tid], wml[2 * tid + 1]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int idx = tid + i * kThreads;
        const int h = idx / (D / 2), d = 2 * (idx - h * (D / 2));
        if (h < G) {
            if constexpr (CLUSTER) {
                store_remote(hand + (h * D + d) * 4, sum[i].x, sum[i].y);
            } else if (A.n_splits == 1) {
                const float inv = s_inv[h];
                *reinterpret_cast<uint32_t *>(A.out + ((size_t)b * A.Hq + h0 + h) * D + d) =
                    pack_bf16x2(sum[i].x * inv, sum[i].y * inv);
            } else {
                *reinterpret_cast<float2 *>(A.ws_o + (row0 + (size_t)h * A.n_splits) * D + d) =
                    sum[i];
            }
        }
    }
    if constexpr (CLUSTER) {
        cluster_arrive();
        cluster_wait();
        if (c != 0) return;
        const int n = (len + A.chunk - 1) / A.chunk;
        const float *got = reinterpret_cast<const float *>(smem);
        constexpr int kFloats = S::kGather / 4;
        for (int idx = tid; idx < G * (D / 2); idx += kThreads) {
            const int h = idx / (D / 2), d = 2 * (idx - h * (D / 2));
            const float *ml = got + kCols * D + 2 * h;
            float M = ml[0];
            for (int i = 1; i < n; ++i) M = fmaxf(M, ml[i * kFloats]);
            float L = 0.f, a0 = 0.f, a1 = 0.f;
            for (int i = 0; i < n; ++i) {
                const float f = ex2((ml[i * kFloats] - M) * A.scale_log2);
                const float2 v = *reinterpret_cast<const float2 *>(got + i * kFloats + h * D + d);
                L = fmaf(f, ml[i * kFloats + 1], L);
                a0 = fmaf(f, v.x, a0);
                a1 = fmaf(f, v.y, a1);
            }
            const float inv = 1.f / L;
            *reinterpret_cast<uint32_t *>(A.out + ((size_t)b * A.Hq + h0 + h) * D + d) =
                pack_bf16x2(a0 * inv, a1 * inv);
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
                       int n_splits, int places, int n_rows, float scale_log2,
                       uint16_t *__restrict__ out) {
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
    if (places) {
        const int B = n_rows / Hq;
        const bool mine = lane < B;
        chunk = even_chunk(mine ? len_or_zero(lens, lane, max_len, Lmax) : 0, mine, B, places);
    }
    const int ns = (len - 1) / chunk + 1;                  // len + chunk may pass 2^31
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
        const float alpha = M == -INFINITY ? 0.f : ex2((M - mn) * scale_log2);
        const float w = lane < n ? ex2((mi.x - mn) * scale_log2) : 0.f;
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
            const float f = sm[w] == -INFINITY ? 0.f : ex2((sm[w] - top) * scale_log2);
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

// How a call is cut: heads per CTA, slots per chunk, chunks of a sequence.
struct Plan {
    int G, n_sub, chunk, n_splits, cluster, places;
    bool wide;                         // at most two CTAs an SM
    int most_splits;                   // n_splits of any shorter max_len, at most
};

// Calls whose CTAs all have a place at once (Plan::wide) ask for so much shared memory that
// an SM takes two, which spreads them evenly: 288 of 1024 slots (18 sequences of 2048) take
// 13.6 us, with three on some SMs 17.7.  In calls of more rounds three an SM hide more latency:
// 256 sequences of 256 .. 2048 slots of 8 KV heads, one chunk each, 85 us against 94 with two,
// 512 of 64 29 against 39.
// A cluster against the form with a second kernel: 1 x 612 slots 3.9 us against 4.5 (and one
// launch less for the host: 5.1 against 7.4), 16 x 600 slots of 8 KV heads 7.7 against 11.7,
// 18 x 2048 13.6 against 17.9.
constexpr int kWideSmem = 100 * 1024;
constexpr int kClusterPlaces = 148 * 2;
constexpr int kClusterLen = 4096;      // longer rows want more than eight chunks
constexpr int kPlaces = 148 * kResident;                   // CTAs resident at once
constexpr int kShare = 8;              // chunks a sequence, at least, to share out by lengths
constexpr double kWaves = 8.0 / 3;                         // chunks for each, see make_plan

Plan make_plan(int B, int Hq, int Hkv, int max_len) {
    Plan P;
    const int g = Hq / Hkv;
    P.n_sub = (g + kCols - 1) / kCols;
    P.G = (g + P.n_sub - 1) / P.n_sub;
    P.n_sub = (g + P.G - 1) / P.G;
    P.cluster = P.places = 0;
    P.wide = false;
    // Few, short rows: one to eight chunks of at least 64 slots, merged within a cluster, as
    // long as all CTAs have a place at once (clusters of eight find only half of them: 32 of
    // them took 8.4 us on 4 x 1000 slots of 8 KV heads, of four 5.5) and long chunks fill
    // the places (96 rows of 4096 slots in 192 CTAs 22.5 us, cut finer 18.3).
    const long long rows = (long long)B * Hkv * P.n_sub;
    if (max_len <= kClusterLen && rows <= kClusterPlaces) {
        int c = 1;
        while (c < kMaxCluster && 64 * c < max_len &&
               2 * c * rows <= (2 * c < 8 ? kClusterPlaces : kClusterPlaces / 2))
            c *= 2;
        P.chunk = ((max_len + c - 1) / c + 63) / 64 * 64;
        P.n_splits = (max_len + P.chunk - 1) / P.chunk;
        P.cluster = c > 1 ? c : 0;                         // one chunk needs none
        P.most_splits = 1;             // (shorter calls merge this way too: nothing in memory)
        P.wide = P.chunk <= 1024 || 8 * c * rows >= 7 * kClusterPlaces;
        if (P.wide) return P;
        P.cluster = 0;
    }
    // Few rows: one chunk for each place a CTA can have, shared out by the lengths on the
    // device, so that no place is idle when sequences differ or are far from max_len.  24 / 8
    // heads, D = 128, max_len 65536: 4 sequences of 47179 .. 64169 slots take 57.0 us against
    // 62.6 with the chunks below, one of 65536 and three of 10 23.9 against 28.6, 4 of 2000
    // 9.5 against 15.8, 4 of 65536 68.7 against 66.5; 6 of 16384 .. 32768 47.4 against 54.1.
    // With fewer than kShare chunks a sequence their lengths fit the places badly: 8 of
    // 18646 .. 25728 take 60.3 against 56.4.  Two chunks for each place: 58.4, 26.1, 10.7, 68.7.
    const long long share = kPlaces / ((long long)Hkv * P.n_sub);
    const int most = (int)((max_len + 63LL) / 64);         // chunks of a sequence
    // The chunks below have at least floor(slots / places) slots, and 64: a sequence has
    // no more of them than this, at any length.
    const double even_most = std::ceil(kPlaces * kWaves / (double)rows * (65.0 / 64));
    P.most_splits = even_most < most ? (int)even_most : most;
    if (B <= 32 && kShare * B <= share) {
        const int left = (int)share - B + 1;               // one each to the others
        const int n = most < left ? most : left;
        P.most_splits = n > P.most_splits ? n : P.most_splits;
        if (n > 1 && (long long)B * max_len < (1 << 30)) {
            P.chunk = 64;                                  // the least
            P.places = (int)share;
            P.n_splits = n;
            return P;
        }
    }
    // Longer chunks leave less to start up and merge, shorter ones spread a call evenly
    // over the SMs (sequences shorter than max_len leave theirs out): kWaves chunks for
    // each place a CTA can have, of at least 64 slots.  64 sequences of 256 .. 2048 slots
    // take 28.7 us at 2.7 of them, 30.2 at 4, 31.2 at 5.3, 29.3 at 1; 8 of 18646 .. 32768
    // 53.0, 58.0, 58.1, 62.5.
    const long long slots = rows * max_len;
    const long long even = ((long long)((double)slots / (kPlaces * kWaves)) + 63) / 64 * 64;
    P.chunk = (int)(even < 64 ? 64 : even > 64LL * most ? 64LL * most : even);
    P.n_splits = (max_len - 1) / P.chunk + 1;
    return P;
}

// Partials of that many chunks a row; the outputs start on a 16-byte boundary.
size_t workspace_bytes(int B, int Hq, int D, int n_splits) {
    if (n_splits == 1) return 16;                          // no second kernel: not used
    const size_t rows = (size_t)B * Hq * n_splits;
    return (rows * 2 * 4 + 15) / 16 * 16 + rows * (size_t)D * 4;
}

template <int D, bool CLUSTER>
cudaError_t launch_split(const DecQ4Args &A, bool wide, cudaStream_t s) {
    using S = DecQ4Shape<D>;
    auto kern = decode_q4_kernel<D, CLUSTER>;
    static_assert(kWideSmem >= S::kSmem, "rings");
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = (unsigned)A.cluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = A.places ? dim3(A.Hkv * A.n_sub, 1, A.places)
                           : dim3(A.Hkv * A.n_sub, A.B, CLUSTER ? A.cluster : A.n_splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = wide ? kWideSmem : S::kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    // The kernel's limit of shared memory is raised once per device; a context that does
    // not know of it yet refuses the launch.
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (raised.load(std::memory_order_relaxed) & bit) {
        e = cudaLaunchKernelEx(&cfg, kern, A);
        if (e != cudaErrorInvalidValue) return e;
        cudaGetLastError();
    }
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem);
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
    return cudaLaunchKernelEx(&cfg, kern, A);
}

template <int D>
cudaError_t launch_decode(const DecQ4Args &A, bool wide, cudaStream_t s) {
    if (A.cluster) return launch_split<D, true>(A, wide, s);
    const cudaError_t e = launch_split<D, false>(A, wide, s);
    if (e != cudaSuccess || A.n_splits == 1) return e;
    // One warp a row while a group covers its chunks; four beyond that (65536 slots of one KV
    // head, 342 chunks: 12.2 us a call against 19.9 with one; 55 chunks: 23.2 against 23.9).
    const int rows = A.B * A.Hq;
    auto merge = [&](auto kern, int grid) {
        return launch_pdl(kern, dim3((unsigned)grid), 128, s, (const float *)A.ws_ml,
                          (const float *)A.ws_o, A.lens, A.max_len, A.Hq, A.Lmax, A.chunk,
                          A.n_splits, A.places, rows, A.scale_log2, A.out);
    };
    return A.n_splits > 32 ? merge(decode_q4_merge_kernel<D, 4>, rows)
                           : merge(decode_q4_merge_kernel<D, 1>, (rows + 3) / 4);
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
    const auto kern = D == 64   ? gqa::read_q4_kernel<64>
                      : D == 96 ? gqa::read_q4_kernel<96>
                                : gqa::read_q4_kernel<128>;
    const dim3 grid((unsigned)((Lout - 1) / gqa::kReadRows + 1), Hkv, B);
    const cudaError_t e = gqa::launch_pdl(kern, grid, gqa::kThreads, s, A);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

extern "C" size_t gqa_decode_q4_workspace_bytes(int B, int Hq, int Hkv, int D, int max_len) {
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || max_len < 1 || !gqa_host::head_dim_ok(D))
        return 0;
    return gqa::workspace_bytes(B, Hq, D, gqa::make_plan(B, Hq, Hkv, max_len).most_splits);
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
    const gqa::Plan P = gqa::make_plan(B, Hq, Hkv, max_len_host);
    if (!ws || !aligned16(ws) ||
        ws_bytes < gqa::workspace_bytes(B, Hq, D, P.cluster ? 1 : P.n_splits))
        return GQA_ERR_WORKSPACE;
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
    A.chunk = P.chunk;
    A.cluster = P.cluster;
    A.places = P.places;
    A.n_sub = P.n_sub;
    A.G = P.G;
    A.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)D)) * 1.4426950408889634f * 0x1p69f;
    A.slack = gqa::kSlack / A.scale_log2;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 64   ? gqa::launch_decode<64>(A, P.wide, s)
                          : D == 96 ? gqa::launch_decode<96>(A, P.wide, s)
                                    : gqa::launch_decode<128>(A, P.wide, s);
    return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}
