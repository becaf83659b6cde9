// pkv_decode_int.cuh -- decode attention over integer-coded KV pools, dense and
// over a list of selected blocks.
//
// With key t held as z_t + s_t n_t (n_t the row's codes) and value t as
// z'_t + s'_t n'_t,
//     q . k_t  = s_t (q . n_t) + z_t sum(q)
//     sum_t p_t v_t = sum_t (p_t s'_t) n'_t + sum_t p_t z'_t
// so the codes enter the matrix products as they lie and the parameters are
// applied to 16 scores and 16 probabilities a block, not to 32 D elements.
//
// The products of a 16-token block run on the warp-level tensor-core MMA with
// the G query heads of a KV head on its N = 8 columns, as in
// pkv_decode_mma.cuh (a tile of 8 rows would leave the 5th-generation MMA's
// M >= 64 seven eighths empty, and this path is bound by HBM and by the
// instructions that unpack codes, not by the tensor pipe).  Head groups of one
// run here too: the unpacking, not the product, is the cost per element, and the
// MMA takes two unpacked elements a register where FMAs would take one and a
// conversion.
//
// Unpacking: an f16 whose exponent bits are zero is the integer of its mantissa
// bits times 2^-24, exactly, and the MMA takes such values at full rate.  So a
// code needs no conversion: `word & 0x00ff00ff` is two 8-bit codes as an f16
// pair, `word & 0x000f000f` two 4-bit codes, `word & 0x00f000f0` two more, times
// 16.  2^24 joins the score scale and the output scale, the 16 the query (keys)
// or the odd rows of the output (values).  One logic operation gives two
// elements; 4 bits need a shift per eight.  The tile's byte order (pkv_int.cuh)
// makes the pairs lie along the contraction axis in both products.
//
// The query is scaled by a power of two per head so that its largest element
// is in [2^9, 2^10): every bf16 element above 2^-23 of it keeps all its bits as
// f16.  p_t s'_t enters as an f16 head plus tail (two MMAs), 22 significant
// bits, against a power of two that follows the largest s' the warp has seen.
#pragma once

#include "pkv_decode_mma.cuh"
#include "pkv_int.cuh"

namespace pkv {

template <int D, int BITS>
struct IntCfg {
    using L = IntTile<D, BITS>;
    static constexpr int kWarps = 4;
    static constexpr int kStages = 2;
    static constexpr int kCtasPerSm = 4;
    static constexpr int kStage = 4 * L::kBytes;  // two blocks: K, V, K, V
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kBarOffset = kRing;
    static constexpr int kInfoOffset = kBarOffset + kWarps * kStages * 8;  // valid tokens of a stage's two blocks
    static constexpr int kMergeOffset = kInfoOffset + kWarps * kStages * 8;
    static constexpr int kBytes = kMergeOffset + (kWarps * 8 + 16) * 4 + 128;  // + alignment slack
    static constexpr int kState = (24 + 4 * (D / 16) * 33) * 4;  // a warp's state for the cross-warp merge
    static_assert(kState <= kStages * kStage, "the merge state reuses the warp's ring");
    static_assert(kCtasPerSm * (kBytes + 1024) <= 228 * 1024 || BITS == 8, "residency");
};

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}

// This lane's code words of a row (keys) or of a token pair (values): NW 32-bit words.
template <int NW, int SECOND>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t* w) {
    if constexpr (NW == 2) {
        const uint2 a = lds64(addr);
        w[0] = a.x;
        w[1] = a.y;
    } else {
        const uint4 a = lds128(addr);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        if constexpr (NW == 8) {
            const uint4 b = lds128(addr + SECOND);
            w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        }
    }
}

// f16 pair of codes from a word's even bytes (8 bits) or low halves (4 bits) ...
template <int BITS>
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
    return w & (BITS == 8 ? 0x00ff00ffu : 0x000f000fu);
}
// ... and from its odd bytes, or its high halves (there times 16).
template <int BITS>
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
    return BITS == 8 ? __byte_perm(w, 0u, 0x4341) : w & 0x00f000f0u;
}

template <int D, int BITS, bool SPARSE>
__global__ void __launch_bounds__(128, IntCfg<D, BITS>::kCtasPerSm)
    decode_int_kernel(const DecodeParams p, const int G, const int q_bf16) {
    using C = IntCfg<D, BITS>;
    using L = IntTile<D, BITS>;
    constexpr int NW = C::kWarps, NST = C::kStages, TB = L::kBytes, STAGE = C::kStage;
    constexpr int KS = D / 16;             // k-steps of S = K Q^T and m-tiles of O^T = V^T P^T
    constexpr int WORDS = L::RB / 16;      // code words a lane reads of a row (keys) or half a pair
    constexpr int PER = KS / WORDS;        // MMAs a word feeds: 1 (8 bits) or 2 (4 bits)
    static_assert(WORDS * PER == KS && (PER == 1 || PER == 2), "fragment split");

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128 - (smem_addr(smem_raw) & 127)) & 127);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, qd = lane & 3;
    allow_dependent_launch();
    const int part = blockIdx.x, h = blockIdx.y, s = blockIdx.z;

    int len = __ldg(p.seq_lens + s);
    const int cap = p.MB * kBlockSize;
    bool bad = len < 0 || len > cap;
    len = len < 0 ? 0 : (len > cap ? cap : len);
    int nblk, j0;  // blocks (or list entries) of this partition, its first
    if constexpr (SPARSE) {
        const int per = p.P / kBlockSize;
        j0 = part * per;
        nblk = min(per, p.nsel - j0);
        if (bad && threadIdx.x == 0 && part == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
    } else {
        if (len > p.NP * p.P) {
            bad = true;
            len = p.NP * p.P;
        }
        if (bad && threadIdx.x == 0 && part == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
        const int nparts = len > 0 ? (len + p.P - 1) / p.P : 1;
        if (part >= nparts) return;
        j0 = part * (p.P / kBlockSize);
        nblk = (min(len, (part + 1) * p.P) + kBlockSize - 1) / kBlockSize - j0;
    }
    // a step is two blocks; warp w takes steps w, w + NW, ...
    const int nstep = (nblk + 1) / 2;
    const int ns_w = warp < nstep ? (nstep - warp + NW - 1) / NW : 0;

    unsigned char* ring = smem + warp * NST * STAGE;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOffset) + warp * NST;
    volatile int* info = reinterpret_cast<int*>(smem + C::kInfoOffset) + warp * NST * 2;
    const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.MB;
    const int32_t* list = SPARSE ? p.selected + (static_cast<int64_t>(s) * p.Hkv + h) * p.nsel + j0 : nullptr;
    const unsigned char* kpool = static_cast<const unsigned char*>(p.k_cache);
    const unsigned char* vpool = static_cast<const unsigned char*>(p.v_cache);
    const uint64_t pol = policy_evict_first();
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < NST; ++i) mbar_init(&bars[i], 1);
        mbar_init_fence();
    }
    __syncwarp();

    // Lane 2k + u of (tbl, val) holds the physical block and the valid tokens of
    // block u of this warp's step (window + k), 16 steps a window.
    int tbl = -1, val = 0, k_issue = 0;
    auto issue_next = [&](const int stage) {  // warp-uniform; stage = k_issue % NST
        if ((k_issue & 15) == 0) {
            const int k = k_issue + (lane >> 1);
            const int j = 2 * (warp + k * NW) + (lane & 1);
            tbl = -1;
            val = 0;
            if (k < ns_w && j < nblk) {
                if constexpr (SPARSE) {
                    tbl = sparse_block(p, s, __ldg(list + j), len, val);
                } else {
                    tbl = __ldg(table + j0 + j);
                    val = min(kBlockSize, len - (j0 + j) * kBlockSize);
                }
                if (val > 0 && (tbl < 0 || tbl >= p.NB)) {
                    report(p.err, PKV_DEVERR_BLOCK_ID);
                    val = 0;
                }
            }
        }
        const int at = 2 * (k_issue & 15);
        const int b0 = __shfl_sync(kFull, tbl, at), b1 = __shfl_sync(kFull, tbl, at + 1);
        const int n0 = __shfl_sync(kFull, val, at), n1 = __shfl_sync(kFull, val, at + 1);
        if (lane == 0) {
            info[2 * stage] = n0;
            info[2 * stage + 1] = n1;
            unsigned char* dst = ring + stage * STAGE;
            mbar_arrive_expect_tx(&bars[stage], (n0 > 0 ? 2 * TB : 0) + (n1 > 0 ? 2 * TB : 0));
            if (n0 > 0) {
                const int64_t off = (static_cast<int64_t>(b0) * p.Hkv + h) * TB;
                bulk_g2s(dst, kpool + off, TB, &bars[stage], pol);
                bulk_g2s(dst + TB, vpool + off, TB, &bars[stage], pol);
            }
            if (n1 > 0) {
                const int64_t off = (static_cast<int64_t>(b1) * p.Hkv + h) * TB;
                bulk_g2s(dst + 2 * TB, kpool + off, TB, &bars[stage], pol);
                bulk_g2s(dst + 3 * TB, vpool + off, TB, &bars[stage], pol);
            }
        }
        ++k_issue;
    };
#pragma unroll
    for (int i = 0; i < NST; ++i)
        if (k_issue < ns_w) issue_next(i);

    // ---- B fragments of Q^T (column n = head g8), per-head scale and sum
    uint32_t qb[KS][2];
    float sfA, sfB, qsA, qsB;  // heads 2 qd (A) and 2 qd + 1 (B)
    {
        float f[KS][4];  // the lane's elements in MMA order: b0 = (0, 1), b1 = (2, 3)
        const bool live = g8 < G;
        const unsigned char* row =
            static_cast<const unsigned char*>(p.q) + (static_cast<int64_t>(s) * p.Hq + h * G + (live ? g8 : 0)) * D * 2;
        float amax = 0.f, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WORDS; ++w) {
            // the 32 / BITS elements of the lane's word w start at d0
            const int d0 = BITS == 8 ? 64 * (w >> 2) + 16 * qd + 4 * (w & 3) : (D / 4) * qd + 8 * w;
            float e[32 / BITS];
#pragma unroll
            for (int i = 0; i < 16 / BITS; ++i) {  // 32-bit words of q
                const uint32_t x = live ? __ldg(reinterpret_cast<const uint32_t*>(row + d0 * 2) + i) : 0u;
                if (q_bf16)
                    Unpack<BF16, 2>::run(&x, e + 2 * i);
                else
                    Unpack<F16, 2>::run(&x, e + 2 * i);
            }
#pragma unroll
            for (int i = 0; i < 32 / BITS; ++i) {
                amax = fmaxf(amax, fabsf(e[i]));
                sum += e[i];
            }
            if constexpr (BITS == 8) {
                f[w][0] = e[0]; f[w][1] = e[2]; f[w][2] = e[1]; f[w][3] = e[3];
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f[2 * w + j][0] = e[2 * j];
                    f[2 * w + j][1] = e[2 * j + 4];
                    f[2 * w + j][2] = e[2 * j + 1];
                    f[2 * w + j][3] = e[2 * j + 5];
                }
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        // 2^e with amax * 2^e in [2^9, 2^10), kept within 2^+-100
        const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        const int e = min(max(9 - ex, -100), 100);
        const float up = __int_as_float((e + 127) << 23);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const float hi = BITS == 8 ? up : up * 0.0625f;  // odd elements of 4-bit words come times 16
            qb[i][0] = pack2<false>(f[i][0] * up, f[i][1] * up);
            qb[i][1] = pack2<false>(f[i][2] * hi, f[i][3] * hi);
        }
        const float sf = p.qk_scale * (__int_as_float((127 - e) << 23) * 0x1p24f), qs = p.qk_scale * sum;
        sfA = __shfl_sync(kFull, sf, 8 * qd);
        sfB = __shfl_sync(kFull, sf, 8 * qd + 4);
        qsA = __shfl_sync(kFull, qs, 8 * qd);
        qsB = __shfl_sync(kFull, qs, 8 * qd + 4);
    }

    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mA = -INFINITY, mB = -INFINITY, lA = 0.f, lB = 0.f, zA = 0.f, zB = 0.f;
    uint32_t vref = 0u;  // bits of the power of two that the value scales are taken against
    float vinv = 0.f;

    // the lane's fragment offsets in a tile
    const uint32_t koff = g8 * L::KW + qd * (L::KW / 4);
    const uint32_t voff = WORDS == 2 ? (g8 >> 2) * 256 + qd * 32 + (g8 & 3) * 8
                                     : (g8 >> 1) * 256 + qd * 32 + (g8 & 1) * 16;
    const uint32_t poff = L::kCodes + g8 * 8;
    bool aborted = false;
    uint32_t phase = 0;
    for (int k0 = 0; k0 < ns_w && !aborted; k0 += NST) {
#pragma unroll
        for (int st = 0; st < NST; ++st) {
            if (k0 + st >= ns_w) break;
            if (!mbar_wait(&bars[st], phase)) {
                if (lane == 0) report(p.err, PKV_DEVERR_TIMEOUT);
                aborted = true;
                break;
            }
            const int nv[2] = {info[2 * st], info[2 * st + 1]};
            if (nv[0] + nv[1] > 0) {
                const uint32_t base = smem_addr(ring + st * STAGE);
                const bool whole = nv[0] == kBlockSize && nv[1] == kBlockSize;
                float sv[2][4];  // (token g8, heads A, B), (token g8 + 8, heads A, B)
                float vs[2][2];  // value scale of tokens g8, g8 + 8
                float vz[2][2];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t kt = base + b * 2 * TB;
                    float sa[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                    uint32_t w0[WORDS], w1[WORDS];
                    lds_words<WORDS, 16 * L::KW>(kt + koff, w0);
                    lds_words<WORDS, 16 * L::KW>(kt + koff + 8 * L::KW, w1);
                    const uint2 kp0 = lds64(kt + poff), kp1 = lds64(kt + poff + 64);
                    const uint2 vp0 = lds64(kt + TB + poff), vp1 = lds64(kt + TB + poff + 64);
#pragma unroll
                    for (int w = 0; w < WORDS; ++w)
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const uint32_t x = w0[w] >> (8 * j), y = w1[w] >> (8 * j);
                            mma16816a<false>(sa[(w * PER + j) & 1], codes_lo<BITS>(x), codes_lo<BITS>(y),
                                             codes_hi<BITS>(x), codes_hi<BITS>(y), qb[w * PER + j][0],
                                             qb[w * PER + j][1]);
                        }
                    const float ks0 = __uint_as_float(kp0.x), ks1 = __uint_as_float(kp1.x);
                    const float kz0 = __uint_as_float(kp0.y), kz1 = __uint_as_float(kp1.y);
                    sv[b][0] = fmaf(ks0 * (sa[0][0] + sa[1][0]), sfA, kz0 * qsA);
                    sv[b][1] = fmaf(ks0 * (sa[0][1] + sa[1][1]), sfB, kz0 * qsB);
                    sv[b][2] = fmaf(ks1 * (sa[0][2] + sa[1][2]), sfA, kz1 * qsA);
                    sv[b][3] = fmaf(ks1 * (sa[0][3] + sa[1][3]), sfB, kz1 * qsB);
                    vs[b][0] = __uint_as_float(vp0.x);
                    vs[b][1] = __uint_as_float(vp1.x);
                    vz[b][0] = __uint_as_float(vp0.y);
                    vz[b][1] = __uint_as_float(vp1.y);
                    if (!whole) {  // tokens past the end: stale parameters must not get through
                        if (g8 >= nv[b]) {
                            sv[b][0] = sv[b][1] = -INFINITY;
                            vs[b][0] = vz[b][0] = 0.f;
                        }
                        if (g8 + 8 >= nv[b]) {
                            sv[b][2] = sv[b][3] = -INFINITY;
                            vs[b][1] = vz[b][1] = 0.f;
                        }
                    }
                }
                float bA = fmaxf(fmaxf(sv[0][0], sv[0][2]), fmaxf(sv[1][0], sv[1][2]));
                float bB = fmaxf(fmaxf(sv[0][1], sv[0][3]), fmaxf(sv[1][1], sv[1][3]));
#pragma unroll
                for (int mask = 4; mask < 32; mask <<= 1) {
                    bA = fmaxf(bA, __shfl_xor_sync(kFull, bA, mask));
                    bB = fmaxf(bB, __shfl_xor_sync(kFull, bB, mask));
                }
                // lazy reference maximum, as in pkv_decode_mma.cuh
                const bool rbA = bA > mA + kRebaseLog2, rbB = bB > mB + kRebaseLog2;
                const float nA = rbA ? bA : mA, nB = rbB ? bB : mB;
                float alA = rbA ? ex2(mA - nA) : 1.f, alB = rbB ? ex2(mB - nB) : 1.f;
                mA = nA;
                mB = nB;
                lA *= alA;
                lB *= alB;
                zA *= alA;
                zB *= alB;
                // the value scales' reference moves only up, by powers of two
                const uint32_t vmax = __reduce_max_sync(
                    kFull, __float_as_uint(fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]))));
                bool move = vmax >= vref;
                if (__builtin_expect(__any_sync(kFull, rbA || rbB || move), 0)) {
                    if (move) {
                        const uint32_t next = (min(vmax >> 23, 251u) + 1u) << 23;
                        const float inv = __uint_as_float((254u << 23) - next);
                        const float f = __uint_as_float(vref) * inv;  // 0 on the first block
                        vref = next;
                        vinv = inv;
                        alA *= f;
                        alB *= f;
                    }
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[i][0] *= alA;
                        o[i][1] *= alB;
                        o[i][2] *= alA;
                        o[i][3] *= alB;
                    }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t vt = base + (2 * b + 1) * TB;
                    const float p0 = ex2(sv[b][0] - nA), p1 = ex2(sv[b][1] - nB);
                    const float p2 = ex2(sv[b][2] - nA), p3 = ex2(sv[b][3] - nB);
                    lA += p0 + p2;
                    lB += p1 + p3;
                    zA = fmaf(p0, vz[b][0], fmaf(p2, vz[b][1], zA));
                    zB = fmaf(p1, vz[b][0], fmaf(p3, vz[b][1], zB));
                    const float u0 = vs[b][0] * vinv, u1 = vs[b][1] * vinv;
                    uint32_t h01, t01, h23, t23;
                    pack2_split<false>(p0 * u0, p1 * u0, h01, t01);
                    pack2_split<false>(p2 * u1, p3 * u1, h23, t23);
                    const uint32_t pb0 = movmatrix_t(h01), pt0 = movmatrix_t(t01);  // tokens 0..7
                    const uint32_t pb1 = movmatrix_t(h23), pt1 = movmatrix_t(t23);  // tokens 8..15
                    uint32_t w0[WORDS], w1[WORDS];
                    lds_words<WORDS, 1024>(vt + voff, w0);
                    lds_words<WORDS, 1024>(vt + voff + 128, w1);
#pragma unroll
                    for (int w = 0; w < WORDS; ++w)
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const uint32_t x = w0[w] >> (8 * j), y = w1[w] >> (8 * j);
                            const uint32_t a0 = codes_lo<BITS>(x), a1 = codes_hi<BITS>(x);
                            const uint32_t a2 = codes_lo<BITS>(y), a3 = codes_hi<BITS>(y);
                            mma16816a<false>(o[w * PER + j], a0, a1, a2, a3, pb0, pb1);
                            mma16816a<false>(o[w * PER + j], a0, a1, a2, a3, pt0, pt1);
                        }
                }
            }
            __syncwarp();
            if (k_issue < ns_w) issue_next(st);
        }
        phase ^= 1u;
    }
    if (aborted) {  // let copies in flight land before the ring is reused
        for (int k = 0; k < NST; ++k) {
            const int kk = k_issue - 1 - k;
            if (kk < 0) break;
            (void)mbar_wait(&bars[kk % NST], (kk / NST) & 1);
        }
    }

    // ---- warp state: [8] m, [8] l, [8] z, then the accumulators in value units,
    // fragment order, 33-word pitch
#pragma unroll
    for (int mask = 4; mask < 32; mask <<= 1) {
        lA += __shfl_xor_sync(kFull, lA, mask);
        lB += __shfl_xor_sync(kFull, lB, mask);
        zA += __shfl_xor_sync(kFull, zA, mask);
        zB += __shfl_xor_sync(kFull, zB, mask);
    }
    float* ws = reinterpret_cast<float*>(ring);
    __syncwarp();
    if (g8 == 0) {
        ws[2 * qd] = aborted ? -INFINITY : mA;
        ws[2 * qd + 1] = aborted ? -INFINITY : mB;
        ws[8 + 2 * qd] = aborted ? 0.f : lA;
        ws[8 + 2 * qd + 1] = aborted ? 0.f : lB;
        ws[16 + 2 * qd] = aborted ? 0.f : zA;
        ws[16 + 2 * qd + 1] = aborted ? 0.f : zB;
    }
    const float os = __uint_as_float(vref) * 0x1p24f;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            ws[24 + (4 * i + c) * 33 + lane] =
                aborted ? 0.f : o[i][c] * (c >= 2 && BITS == 4 ? os * 0.0625f : os);
    __syncthreads();

    // ---- cross-warp log-sum-exp weights, once per (warp, head)
    float* msc = reinterpret_cast<float*>(smem + C::kMergeOffset);  // [NW][8]
    float* minv = msc + NW * 8;
    float* mmax = minv + 8;
    if (threadIdx.x < G) {
        const int g = threadIdx.x;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) M = fmaxf(M, reinterpret_cast<float*>(smem + w * NST * STAGE)[g]);
        float den = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float* wsw = reinterpret_cast<float*>(smem + w * NST * STAGE);
            const float sc = (M != -INFINITY && wsw[g] != -INFINITY) ? exp2f(wsw[g] - M) : 0.f;
            msc[w * 8 + g] = sc;
            den = fmaf(sc, wsw[8 + g], den);
        }
        minv[g] = den > 0.f ? 1.f / den : (den == den ? 0.f : den);
        mmax[g] = M;
        const int64_t row = static_cast<int64_t>(s) * p.Hq + h * G + g;
        if (p.NP > 1) {
            p.part_m[row * p.NP + part] = M;
            p.part_l[row * p.NP + part] = den;
        }
    }
    __syncthreads();

    // ---- output: element pairs (head g, dimensions d, d + 1) over the threads
    const bool direct = SPARSE ? p.NP == 1 : len <= p.P;
    for (int i2 = threadIdx.x; i2 < G * (D / 2); i2 += NW * 32) {
        const int g = i2 / (D / 2), d = 2 * (i2 % (D / 2));
        // inverse of the fragment layout: m-tile i of lane group gl holds (d, d + 1) in its two row halves
        int i, gl;
        if constexpr (D == 128 && BITS == 8) {
            i = 4 * (d >> 6) + ((d >> 1) & 3);
            gl = (d >> 3) & 7;
        } else {
            i = (d >> 1) % KS;
            gl = d / (2 * KS);
        }
        const int frag = 24 + (4 * i + (g & 1)) * 33 + 4 * gl + (g >> 1);
        float r0 = 0.f, r1 = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float* wsw = reinterpret_cast<float*>(smem + w * NST * STAGE);
            const float sc = msc[w * 8 + g];
            if (sc != 0.f) {
                r0 = fmaf(sc, wsw[frag] + wsw[16 + g], r0);
                r1 = fmaf(sc, wsw[frag + 66] + wsw[16 + g], r1);
            }
        }
        r0 *= minv[g];
        r1 *= minv[g];
        const int64_t row = static_cast<int64_t>(s) * p.Hq + h * G + g;
        if (direct) {
            reinterpret_cast<uint32_t*>(p.out)[(row * D + d) / 2] = q_bf16 ? pack2<true>(r0, r1) : pack2<false>(r0, r1);
        } else {
            *reinterpret_cast<float2*>(p.part_o + (row * p.NP + part) * D + d) = make_float2(r0, r1);
        }
    }
}

template <int D, int BITS, bool SPARSE>
cudaError_t launch_decode_int_t(const DecodeParams& p, int G, int q_dtype, cudaStream_t st) {
    constexpr int SMEM = IntCfg<D, BITS>::kBytes;
    auto kern = decode_int_kernel<D, BITS, SPARSE>;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    kern<<<dim3(p.NP, p.Hkv, p.S), 128, SMEM, st>>>(p, G, q_dtype == PKV_BF16 ? 1 : 0);
    return cudaGetLastError();
}

template <int BITS>
cudaError_t launch_decode_int(const DecodeParams& p, int G, int q_dtype, cudaStream_t st) {
    if (p.selected)
        return p.D == 128 ? launch_decode_int_t<128, BITS, true>(p, G, q_dtype, st)
                          : launch_decode_int_t<64, BITS, true>(p, G, q_dtype, st);
    return p.D == 128 ? launch_decode_int_t<128, BITS, false>(p, G, q_dtype, st)
                      : launch_decode_int_t<64, BITS, false>(p, G, q_dtype, st);
}

}  // namespace pkv
