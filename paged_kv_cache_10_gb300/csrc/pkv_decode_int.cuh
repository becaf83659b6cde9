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
// elements; 4 bits need a byte shuffle per eight.  The tile's byte order (pkv_int.cuh)
// makes the pairs lie along the contraction axis in both products.
//
// The query is scaled by a power of two per head so that its largest element
// is in [2^9, 2^10), and enters as f16: an element loses bits only below 2^-19 of
// that (2^-22 from bf16), where a step is 2^-30 of the largest.  p_t s'_t enters
// as an f16 head plus tail, scaled by a power of two c per head that follows the
// largest p_t s'_t of the head's rows so far (kept between 2^6 and 2^15, so that
// the pair's steps, 22 significant bits or 2^-25, are at most 2^-31 of it): a row
// of a wide range that the query does not attend to takes no bits of the others.
// Two MMAs, or one for groups of up to four heads, whose tails ride in the spare
// columns 4 .. 7 (64 x U[512, 4096] 32/32 heads, int4, when it was taken: 135.7 ->
// 128.5 us).
//
// A warp's step is two blocks: one barrier wait, one vote and one load of Q's
// fragments for 32 tokens, and two independent chains of MMAs.  A ring of two steps
// a warp and 16 warps an SM (12 for 8 bits at D = 128, by shared memory) keep 140 to
// 210 KB of copies in flight; a third step, a fifth CTA (96 registers, which
// spill) and CTAs of 2, 3 or 8 warps measured slower.
//
// Measured on one GB300 (calls replayed in a graph, share of the measured HBM copy
// bandwidth on the bytes the call cannot do without): int8 256 x U[128, 2048],
// 32/8 heads 96.3 us (0.98); int8 64 x U[512, 4096], 32/32 heads 187 us (1.04);
// int4 8 x 32768, 64/8 heads 58.8 us (0.76); int4 256 x U[128, 2048], 32/8 heads
// 66.1 us (0.72).  8 bits are bound by HBM.  4 bits halve the bytes but not the
// instructions: 243 a block and warp plus 850 a warp for its start and end, issued
// in 54 % of the cycles; with its copies left out an earlier version took 55 of its
// 63 us.  Following the largest p s' costs the 4 bits 1.3 to 2.4 of these us.
#pragma once

#include "pkv_decode_mma.cuh"
#include "pkv_int.cuh"

namespace pkv {

// FOLD: groups of at most four heads, whose columns 4 .. 7 carry the tails.
template <int D, int BITS, bool FOLD>
struct IntCfg {
    using L = IntTile<D, BITS>;
    static constexpr int kWarps = 4;
    static constexpr int kStages = 2;
    static constexpr int kCtasPerSm = BITS == 8 && D == 128 ? 3 : 4;  // as many as shared memory holds
    static constexpr int kStage = 4 * L::kBytes;  // two blocks: K, V, K, V
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kBarOffset = kRing;
    static constexpr int kInfoOffset = kBarOffset + kWarps * kStages * 8;  // valid tokens of a stage's two blocks
    static constexpr int kMergeOffset = kInfoOffset + (kWarps * kStages * 2 + 15) / 16 * 16;
    static constexpr int kQOffset = (kMergeOffset + kWarps * 24 * 4 + 15) / 16 * 16;  // Q^T fragments, 8 bytes a lane and k-step
    static constexpr int kBytes = kQOffset + (D / 16) * 32 * 8 + 128;  // + alignment slack
    static constexpr int kState = 8 * (D + 4) * 4;  // a warp's accumulators for the cross-warp merge
    static_assert(kState <= kStages * kStage, "the merge state reuses the warp's ring");
    static_assert(kCtasPerSm * (kBytes + 1024) <= 228 * 1024, "residency");
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

// The A operand pairs of code word w for its j-th MMA (j = 0 for 8 bits): lo from
// the even bytes or, of byte j of each half, the low codes, hi from the odd bytes
// or the high codes times 16.  The second byte's low codes are what is left of
// the byte without the high ones: a subtraction, exact on these values, that
// runs beside the logic operations instead of among them.
template <int BITS>
__device__ __forceinline__ void code_pairs(uint32_t w, int j, uint32_t& lo, uint32_t& hi) {
    if constexpr (BITS == 8) {
        lo = w & 0x00ff00ffu;
        hi = __byte_perm(w, 0u, 0x4341);
    } else if (j == 0) {
        lo = w & 0x000f000fu;
        hi = w & 0x00f000f0u;
    } else {
        const uint32_t x = __byte_perm(w, 0u, 0x4341);
        hi = x & 0x00f000f0u;
        const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&hi));
        lo = *reinterpret_cast<const uint32_t*>(&d);
    }
}

// 2^e / c for a power of two c, the quotient within binary32's normal range.
__device__ __forceinline__ float pow2_over(int e, float c) {
    return __uint_as_float((static_cast<uint32_t>(254 + e) << 23) - __float_as_uint(c));
}

// Moves a head's scale c of its weights p s' and lim = 2^15 / c, the largest p s' that
// it takes, the softmax maximum having moved by the factor a (1: it stays); y is the
// largest p s' of the step against the new maximum.  The larger of y and of what was
// seen before, taken as 2^6 / c, comes to lie in [2^6, 2^7) / c; c stays within
// 2^+-118, lim below 2^128.  Returns the accumulators' factor.
__device__ __forceinline__ float move_weights(float& c, float& lim, float a, float y) {
    if (a == 1.f && y <= lim) return 1.f;
    const int was = static_cast<int>(__float_as_uint(c) >> 23);
    const float top = fmaxf(y, a * pow2_over(6, c));
    const int now = min(max(127 + 6 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 127 - 118), 127 + 118);
    c = __int_as_float(now << 23);
    lim = __int_as_float(min(127 + 15 + 127 - now, 254) << 23);
    const int d = now - was, half = d >> 1;  // 2^d in two steps: d is within +-236
    return a * __int_as_float((127 + half) << 23) * __int_as_float((127 + d - half) << 23);
}

template <int D, int BITS, bool FOLD, bool SPARSE, bool SCORED>
__global__ void __launch_bounds__(IntCfg<D, BITS, FOLD>::kWarps * 32, IntCfg<D, BITS, FOLD>::kCtasPerSm)
    decode_int_kernel(const DecodeParams p, const int G, const int q_bf16) {
    using C = IntCfg<D, BITS, FOLD>;
    using L = IntTile<D, BITS>;
    constexpr int NW = C::kWarps, NST = C::kStages, TB = L::kBytes, STAGE = C::kStage;
    constexpr int KS = D / 16;             // k-steps of S = K Q^T and m-tiles of O^T = V^T P^T
    constexpr int WORDS = L::RB / 16;      // code words a lane reads of a row (keys) or half a pair
    constexpr int PER = KS / WORDS;        // MMAs a word feeds: 1 (8 bits) or 2 (4 bits)
    constexpr int kGroup = 2;
    static_assert(WORDS * PER == KS && (PER == 1 || PER == 2), "fragment split");

    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128 - (smem_addr(smem_raw) & 127)) & 127);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g8 = lane >> 2, qd = lane & 3;
    const int part = blockIdx.x, h = blockIdx.y, s = blockIdx.z;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOffset) + warp * NST;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < NST; ++i) mbar_init(&bars[i], 1);
        mbar_init_fence();
    }
    // A programmatic dependent of the kernel before it on the stream: what it reads
    // may come from there.  Its own dependent, the merge, reads the lengths before it
    // waits, so it may start only now.
    wait_primary_grid();
    allow_dependent_launch();
    // the first window's table (or list) entries, loaded beside the length
    const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.MB;
    int len;
    bool bad;
    const auto load_len = [&] {
        len = load_live(p.seq_lens + s);
        const int cap = p.MB * kBlockSize;
        bad = len < 0 || len > cap;
        len = len < 0 ? 0 : (len > cap ? cap : len);
    };
    ScoredRow row{};  // scored: the row's range, which its table entries wait for
    if constexpr (SCORED) {
        load_len();
        row = scored_row(p, s, len, bad);
        len = row.end;
        if (bad && threadIdx.x == 0 && part == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
        if (part >= scored_parts(p, row)) return;
    }
    // first block (or list entry) of this partition
    const int j0 = part * (p.P / kBlockSize) + (SCORED ? row.start / kBlockSize : 0);
    const int32_t* list = SPARSE ? p.selected + (static_cast<int64_t>(s) * p.Hkv + h) * p.nsel + j0 : table + j0;
    const int list_len = (SPARSE ? p.nsel : p.MB) - j0;
    const auto entry = [&](int k) {  // lane 2i + u: block u of this warp's step k + i
        const int j = 2 * (warp + (k + (lane >> 1)) * NW) + (lane & 1);
        return j < list_len ? load_live(list + j) : -1;
    };
    int next = entry(0);
    if constexpr (!SCORED) load_len();
    int nblk;  // blocks (or list entries) of this partition
    if constexpr (SPARSE) {
        nblk = min(p.P / kBlockSize, list_len);
        if (bad && threadIdx.x == 0 && part == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
    } else if constexpr (SCORED) {
        nblk = row.lo < len ? (min(len, row.start + (part + 1) * p.P) + kBlockSize - 1) / kBlockSize - j0 : 0;
    } else {
        if (len > p.NP * p.P) {
            bad = true;
            len = p.NP * p.P;
        }
        if (bad && threadIdx.x == 0 && part == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
        const int nparts = len > 0 ? (len + p.P - 1) / p.P : 1;
        if (part >= nparts) return;
        nblk = (min(len, (part + 1) * p.P) + kBlockSize - 1) / kBlockSize - j0;
    }
    // a step is two blocks; warp w takes steps w, w + NW, ...
    const int nstep = (nblk + 1) / 2;
    const int ns_w = warp < nstep ? (nstep - warp + NW - 1) / NW : 0;

    unsigned char* ring = smem + warp * NST * STAGE;
    volatile unsigned char* info = smem + C::kInfoOffset + warp * NST * 2;
    const unsigned char* kpool = static_cast<const unsigned char*>(p.k_cache);
    const unsigned char* vpool = static_cast<const unsigned char*>(p.v_cache);
    const uint64_t pol = policy_evict_first();
    __syncwarp();

    // Lane 2k + u of (tbl, val) holds the physical block and the valid tokens of
    // block u of this warp's step (window + k), 16 steps a window.
    int tbl = -1, val = 0, k_issue = 0;
    auto issue_next = [&](const int stage) {  // warp-uniform; stage = k_issue % NST
        if ((k_issue & 15) == 0) {
            const int k = k_issue + (lane >> 1);
            const int j = 2 * (warp + k * NW) + (lane & 1);
            const int e = next;
            tbl = -1;
            val = 0;
            if (k < ns_w && j < nblk) {
                if constexpr (SPARSE) {
                    tbl = sparse_block(p, s, e, len, val);
                } else {
                    tbl = e;
                    val = min(kBlockSize, len - (j0 + j) * kBlockSize);
                }
                if (val > 0 && (tbl < 0 || tbl >= p.NB)) {
                    report(p.err, PKV_DEVERR_BLOCK_ID);
                    val = 0;
                }
            }
            next = entry(k_issue + 16);  // a window ahead
        }
        // the two lanes that hold the step's blocks issue their copies
        const uint32_t both = __ballot_sync(kFull, val > 0) >> (2 * (k_issue & 15)) & 3u;
        const int u = lane - 2 * (k_issue & 15);
        if (u == 0) mbar_arrive_expect_tx(&bars[stage], __popc(both) * 2 * TB);
        __syncwarp();
        if (u == 0 || u == 1) {
            info[2 * stage + u] = static_cast<unsigned char>(val);
            if (val > 0) {
                unsigned char* dst = ring + stage * STAGE + u * 2 * TB;
                // tiles of a pool count below 2^32
                const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(tbl) * static_cast<uint32_t>(p.Hkv) + h) * TB;
                bulk_g2s(dst, kpool + off, TB, &bars[stage], pol);
                bulk_g2s(dst + TB, vpool + off, TB, &bars[stage], pol);
            }
        }
        ++k_issue;
    };
#pragma unroll
    for (int i = 0; i < NST; ++i)
        if (k_issue < ns_w) issue_next(i);

    // ---- B fragments of Q^T (column n = head g8), per-head scale and sum: the
    // warps share the words, each head's extrema and sums meet in shared memory
    uint2* qsm = reinterpret_cast<uint2*>(smem + C::kQOffset);
    float* msc = reinterpret_cast<float*>(smem + C::kMergeOffset);
    float sfA, sfB, qsA, qsB;  // heads 2 qd (A) and 2 qd + 1 (B)
    {
        constexpr int EPW = 32 / BITS;                // elements of a word
        constexpr int MINE = (WORDS + NW - 1) / NW;   // words a warp takes
        const int head = FOLD ? g8 & 3 : g8;  // FOLD: columns 4 .. 7 repeat the heads
        const bool live = head < G;
        const unsigned char* row =
            static_cast<const unsigned char*>(p.q) + (static_cast<int64_t>(s) * p.Hq + h * G + (live ? head : 0)) * D * 2;
        float e[MINE][EPW];
        float amax = 0.f, sum = 0.f;
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
            const int w = warp + m * NW;
            const int d0 = BITS == 8 ? 64 * (w >> 2) + 16 * qd + 4 * (w & 3) : (D / 4) * qd + 8 * w;
            uint32_t x[EPW / 2];
#pragma unroll
            for (int i = 0; i < EPW / 2; ++i) x[i] = 0u;
            if (live && w < WORDS) load_words<EPW * 2>(row + d0 * 2, x);
            if (q_bf16)
                Unpack<BF16, EPW>::run(x, e[m]);
            else
                Unpack<F16, EPW>::run(x, e[m]);
#pragma unroll
            for (int i = 0; i < EPW; ++i) {
                amax = fmaxf(amax, fabsf(e[m][i]));
                sum += e[m][i];
            }
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        if (qd == 0) reinterpret_cast<float2*>(msc)[warp * 8 + g8] = make_float2(amax, sum);
        __syncthreads();
        amax = sum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float2 v = reinterpret_cast<const float2*>(msc)[w * 8 + g8];
            amax = fmaxf(amax, v.x);
            sum += v.y;
        }
        // 2^ex with amax * 2^ex in [2^9, 2^10); 2^(24 - ex), the scores' factor, stays in binary32's
        // range, so that an element of 2^119 or more becomes infinite and one below 2^-118 loses bits
        const int ex = min(max(9 + 127 - static_cast<int>(__float_as_uint(amax) >> 23), -103), 127);
        const float up = __int_as_float((ex + 127) << 23);
        const float hi = BITS == 8 ? up : up * 0.0625f;  // odd elements of 4-bit words come times 16
#pragma unroll
        for (int m = 0; m < MINE; ++m) {
            const int w = warp + m * NW;
            if (w >= WORDS) break;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                constexpr int R = BITS == 8 ? 2 : 4;  // element distance of an f16 pair
                qsm[(w * PER + j) * 32 + lane] = make_uint2(pack2<false>(e[m][2 * j] * up, e[m][2 * j + R] * up),
                                                            pack2<false>(e[m][2 * j + 1] * hi, e[m][2 * j + 1 + R] * hi));
            }
        }
        const float sf = p.qk_scale * __int_as_float((127 + 24 - ex) << 23), qs = p.qk_scale * sum;
        sfA = __shfl_sync(kFull, sf, 8 * qd);
        sfB = __shfl_sync(kFull, sf, 8 * qd + 4);
        qsA = __shfl_sync(kFull, qs, 8 * qd);
        qsB = __shfl_sync(kFull, qs, 8 * qd + 4);
    }
    __syncthreads();

    float o[KS][4];
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mA = kNoScore, mB = kNoScore, lA = 0.f, lB = 0.f, zA = 0.f, zB = 0.f;
    float cA = 0x1p118f, cB = 0x1p118f, limA = 0x1p-103f, limB = 0x1p-103f;  // scales of the weights p s'

    float slopeA = 0.f, slopeB = 0.f;
    const int colA = FOLD ? 2 * qd & 3 : 2 * qd;  // the lane's heads in the group
    if constexpr (SCORED) {
        if (colA < G) slopeA = scored_slope(p, h * G + colA);
        if (colA + 1 < G) slopeB = scored_slope(p, h * G + colA + 1);
    }

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
            const uint32_t nvs = *reinterpret_cast<const volatile uint16_t*>(info + 2 * st);
            // scored: first token of the step, tokens in front of the row's first
            const int tok0 = SCORED ? (j0 + 2 * (warp + (k0 + st) * NW)) * kBlockSize : 0;
            const int lead = SCORED ? row.lo - tok0 : 0;
            if (nvs != 0u) {
                const uint32_t base = smem_addr(ring + st * STAGE);
                const bool whole = nvs == (kBlockSize << 8 | kBlockSize);
                const int nv[2] = {static_cast<int>(nvs & 255u), static_cast<int>(nvs >> 8)};
                float sv[2][4];  // (token g8, heads A, B), (token g8 + 8, heads A, B)
                float vs[2][2];  // value scale of tokens g8, g8 + 8
                float vz[2][2];
                {
                    // the two blocks' products side by side: two chains of MMAs, one load of Q
                    // for both (two accumulators a block, added at the end: 58.8 us against
                    // 58.0 on 8 x 32768 tokens at 4 bits)
                    float sa[2][4];
                    uint32_t w0[2][WORDS], w1[2][WORDS];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t kt = base + b * 2 * TB + koff;
                        lds_words<WORDS, 16 * L::KW>(kt, w0[b]);
                        lds_words<WORDS, 16 * L::KW>(kt + 8 * L::KW, w1[b]);
                        sa[b][0] = sa[b][1] = sa[b][2] = sa[b][3] = 0.f;
                    }
#pragma unroll
                    for (int w = 0; w < WORDS; ++w)
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const uint2 qf = qsm[(w * PER + j) * 32 + lane];
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                uint32_t a0, a1, a2, a3;
                                code_pairs<BITS>(w0[b][w], j, a0, a2);
                                code_pairs<BITS>(w1[b][w], j, a1, a3);
                                mma16816a<false>(sa[b], a0, a1, a2, a3, qf.x, qf.y);
                            }
                        }
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t kp = base + b * 2 * TB + poff;
                        const uint2 kp0 = lds64(kp), kp1 = lds64(kp + 64);
                        const float ks0 = __uint_as_float(kp0.x), ks1 = __uint_as_float(kp1.x);
                        const float kz0 = __uint_as_float(kp0.y), kz1 = __uint_as_float(kp1.y);
                        sv[b][0] = fmaf(ks0 * sa[b][0], sfA, kz0 * qsA);
                        sv[b][1] = fmaf(ks0 * sa[b][1], sfB, kz0 * qsB);
                        sv[b][2] = fmaf(ks1 * sa[b][2], sfA, kz1 * qsA);
                        sv[b][3] = fmaf(ks1 * sa[b][3], sfB, kz1 * qsB);
                        if constexpr (SCORED) {
                            const int t0 = b * kBlockSize + g8, t1 = t0 + 8;
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                sv[b][c] = scored(p, sv[b][c], (c & 1) ? slopeB : slopeA, row.end - 1 - tok0 - (c < 2 ? t0 : t1));
                            if (t0 < lead) sv[b][0] = sv[b][1] = -INFINITY;
                            if (t1 < lead) sv[b][2] = sv[b][3] = -INFINITY;
                            if (p.scores && (FOLD ? qd < 2 : true)) {
                                // past the row's last block (an odd step) there is no room
                                float* out = p.scores + ((static_cast<int64_t>(s) * p.Hkv + h) * p.span + (tok0 - row.start)) * G;
                                if (t0 < b * kBlockSize + nv[b]) {
                                    if (colA < G) out[t0 * G + colA] = sv[b][0];
                                    if (colA + 1 < G) out[t0 * G + colA + 1] = sv[b][1];
                                }
                                if (t1 < b * kBlockSize + nv[b]) {
                                    if (colA < G) out[t1 * G + colA] = sv[b][2];
                                    if (colA + 1 < G) out[t1 * G + colA + 1] = sv[b][3];
                                }
                            }
                        }
                        if (!whole) {  // tokens past the end: stale parameters must not get through
                            if (g8 >= nv[b]) sv[b][0] = sv[b][1] = -INFINITY;
                            if (g8 + 8 >= nv[b]) sv[b][2] = sv[b][3] = -INFINITY;
                        }
                    }
                }
                float bA = fmaxf(fmaxf(sv[0][0], sv[0][2]), fmaxf(sv[1][0], sv[1][2]));
                float bB = fmaxf(fmaxf(sv[0][1], sv[0][3]), fmaxf(sv[1][1], sv[1][3]));
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint2 vp0 = lds64(base + (2 * b + 1) * TB + poff), vp1 = lds64(base + (2 * b + 1) * TB + poff + 64);
                    vs[b][0] = __uint_as_float(vp0.x);
                    vs[b][1] = __uint_as_float(vp1.x);
                    vz[b][0] = __uint_as_float(vp0.y);
                    vz[b][1] = __uint_as_float(vp1.y);
                    if (!whole) {
                        if (g8 >= nv[b]) vs[b][0] = vz[b][0] = 0.f;
                        if (g8 + 8 >= nv[b]) vs[b][1] = vz[b][1] = 0.f;
                    }
                    if constexpr (SCORED) {
                        if (b * kBlockSize + g8 < lead) vs[b][0] = vz[b][0] = 0.f;
                        if (b * kBlockSize + g8 + 8 < lead) vs[b][1] = vz[b][1] = 0.f;
                    }
                }
                // Lazy references, checked lane by lane: the probabilities' maximum moves when a
                // score passes it by 2^kRebaseLog2, the weights' scale when a weight may pass its
                // limit (bounded by the lane's largest probability times its largest value scale).
                // Steps without a move, nearly all, reduce nothing over the warp but this vote.
                const float vm = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
                const float xA = bA - mA, xB = bB - mB;
                if (__builtin_expect(__any_sync(kFull, xA > kRebaseLog2 || xB > kRebaseLog2 ||
                                                           ex2(xA) * vm > limA || ex2(xB) * vm > limB), 0)) {
#pragma unroll
                    for (int mask = 4; mask < 32; mask <<= 1) {
                        bA = fmaxf(bA, __shfl_xor_sync(kFull, bA, mask));
                        bB = fmaxf(bB, __shfl_xor_sync(kFull, bB, mask));
                    }
                    float alA = 1.f, alB = 1.f;
                    if (bA - mA > kRebaseLog2) {
                        alA = ex2(mA - bA);  // 0 on the first block
                        mA = bA;
                    }
                    if (bB - mB > kRebaseLog2) {
                        alB = ex2(mB - bB);
                        mB = bB;
                    }
                    lA *= alA;
                    lB *= alB;
                    zA *= alA;
                    zB *= alB;
                    float yA = 0.f, yB = 0.f;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        yA = fmaxf(yA, fmaxf(ex2(sv[b][0] - mA) * vs[b][0], ex2(sv[b][2] - mA) * vs[b][1]));
                        yB = fmaxf(yB, fmaxf(ex2(sv[b][1] - mB) * vs[b][0], ex2(sv[b][3] - mB) * vs[b][1]));
                    }
#pragma unroll
                    for (int mask = 4; mask < 32; mask <<= 1) {
                        yA = fmaxf(yA, __shfl_xor_sync(kFull, yA, mask));
                        yB = fmaxf(yB, __shfl_xor_sync(kFull, yB, mask));
                    }
                    alA = move_weights(cA, limA, alA, yA);
                    alB = move_weights(cB, limB, alB, yB);
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
                    const float p0 = ex2(sv[b][0] - mA), p1 = ex2(sv[b][1] - mB);
                    const float p2 = ex2(sv[b][2] - mA), p3 = ex2(sv[b][3] - mB);
                    lA += p0 + p2;
                    lB += p1 + p3;
                    zA = fmaf(p0, vz[b][0], fmaf(p2, vz[b][1], zA));
                    zB = fmaf(p1, vz[b][0], fmaf(p3, vz[b][1], zB));
                    // (p c) s', in this order: a wide row that is not attended to gives 0, not 0 * inf
                    uint32_t h01, t01, h23, t23;
                    pack2_split<false>(p0 * cA * vs[b][0], p1 * cB * vs[b][0], h01, t01);
                    pack2_split<false>(p2 * cA * vs[b][1], p3 * cB * vs[b][1], h23, t23);
                    uint32_t pb0, pb1, pt0 = 0u, pt1 = 0u;  // tokens 0 .. 7, tokens 8 .. 15
                    if constexpr (FOLD) {
                        // columns 4 .. 7 (lanes qd >= 2) hold the same probabilities: they
                        // carry the tails, and one MMA does both
                        pb0 = movmatrix_t(qd < 2 ? h01 : t01);
                        pb1 = movmatrix_t(qd < 2 ? h23 : t23);
                    } else {
                        pb0 = movmatrix_t(h01);
                        pt0 = movmatrix_t(t01);
                        pb1 = movmatrix_t(h23);
                        pt1 = movmatrix_t(t23);
                    }
                    uint32_t w0[WORDS], w1[WORDS];
                    lds_words<WORDS, 1024>(vt + voff, w0);
                    lds_words<WORDS, 1024>(vt + voff + 128, w1);
                    // kGroup m-tiles' head products, then their tails: an accumulator's two
                    // MMAs are not back to back
#pragma unroll
                    for (int i0 = 0; i0 < KS; i0 += kGroup) {
                        uint32_t a[kGroup][4];
#pragma unroll
                        for (int i = 0; i < kGroup; ++i) {
                            const int w = (i0 + i) / PER, j = (i0 + i) % PER;
                            code_pairs<BITS>(w0[w], j, a[i][0], a[i][1]);
                            code_pairs<BITS>(w1[w], j, a[i][2], a[i][3]);
                            mma16816a<false>(o[i0 + i], a[i][0], a[i][1], a[i][2], a[i][3], pb0, pb1);
                        }
#pragma unroll
                        for (int i = 0; i < kGroup && !FOLD; ++i)
                            mma16816a<false>(o[i0 + i], a[i][0], a[i][1], a[i][2], a[i][3], pt0, pt1);
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

    // ---- the warps' states meet: maxima first, then each warp writes its sums and
    // accumulators relative to the CTA's maximum, in value units, as rows [column][D]
    // of its ring, so that the last pass only adds them up
#pragma unroll
    for (int mask = 4; mask < 32; mask <<= 1) {
        lA += __shfl_xor_sync(kFull, lA, mask);
        lB += __shfl_xor_sync(kFull, lB, mask);
        zA += __shfl_xor_sync(kFull, zA, mask);
        zB += __shfl_xor_sync(kFull, zB, mask);
    }
    float2* wm = reinterpret_cast<float2*>(msc);  // [NW][4] maxima of columns 2 qd, 2 qd + 1
    float2* wl = wm + NW * 4;
    float2* wz = wl + NW * 4;
    if (aborted) mA = mB = kNoScore;
    if (g8 == 0) wm[warp * 4 + qd] = make_float2(mA, mB);
    __syncthreads();
    float MA = kNoScore, MB = kNoScore;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float2 m = wm[w * 4 + qd];
        MA = fmaxf(MA, m.x);
        MB = fmaxf(MB, m.y);
    }
    const float scA = aborted ? 0.f : ex2(mA - MA), scB = aborted ? 0.f : ex2(mB - MB);
    if (g8 == 0) {
        wl[warp * 4 + qd] = make_float2(scA * lA, scB * lB);
        wz[warp * 4 + qd] = make_float2(scA * zA, scB * zB);
    }
    constexpr int PW = D + 4;
    {
        // 2^24 sc / c in two factors, neither of which overflows
        const float kA = scA * 0x1p16f, kB = scB * 0x1p16f;
        const float oA = pow2_over(8, cA), oB = pow2_over(8, cB);
        constexpr float odd = BITS == 4 ? 0.0625f : 1.f;  // odd rows of 4-bit words come times 16
        float* ws = reinterpret_cast<float*>(ring) + 2 * qd * PW;
#pragma unroll
        for (int i = 0; i < KS; i += 2) {  // m-tiles i, i + 1 hold four consecutive dimensions from d
            const int d = D == 128 && BITS == 8 ? 8 * g8 + 64 * (i >> 2) + 2 * (i & 3) : 2 * KS * g8 + 2 * i;
            *reinterpret_cast<float4*>(ws + d) =
                make_float4(o[i][0] * kA * oA, o[i][2] * (kA * odd) * oA, o[i + 1][0] * kA * oA, o[i + 1][2] * (kA * odd) * oA);
            *reinterpret_cast<float4*>(ws + PW + d) =
                make_float4(o[i][1] * kB * oB, o[i][3] * (kB * odd) * oB, o[i + 1][1] * kB * oB, o[i + 1][3] * (kB * odd) * oB);
        }
    }
    __syncthreads();

    // ---- output: four dimensions of a head a thread
    const bool direct = SPARSE ? p.NP == 1 : SCORED ? !p.cascade && len - row.start <= p.P : len <= p.P;
    for (int i4 = threadIdx.x; i4 < G * (D / 4); i4 += NW * 32) {
        const int g = i4 / (D / 4), d = 4 * (i4 % (D / 4));
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f, z = 0.f, M = kNoScore;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float* x = reinterpret_cast<const float*>(smem + w * NST * STAGE) + g * PW + d;
            const float4 u = *reinterpret_cast<const float4*>(x);
            r.x += u.x; r.y += u.y; r.z += u.z; r.w += u.w;
            if constexpr (FOLD) {  // the tails' columns
                const float4 v = *reinterpret_cast<const float4*>(x + 4 * PW);
                r.x += v.x; r.y += v.y; r.z += v.z; r.w += v.w;
            }
            M = fmaxf(M, msc[w * 8 + g]);
            den += msc[(NW + w) * 8 + g];
            z += msc[(2 * NW + w) * 8 + g];
        }
        const float inv = den > 0.f ? 1.f / den : (den == den ? 0.f : den);
        r = make_float4((r.x + z) * inv, (r.y + z) * inv, (r.z + z) * inv, (r.w + z) * inv);
        const int64_t row = static_cast<int64_t>(s) * p.Hq + h * G + g;
        if (direct) {
            reinterpret_cast<uint2*>(p.out)[(row * D + d) / 4] =
                q_bf16 ? make_uint2(pack2<true>(r.x, r.y), pack2<true>(r.z, r.w))
                       : make_uint2(pack2<false>(r.x, r.y), pack2<false>(r.z, r.w));
        } else {
            *reinterpret_cast<float4*>(p.part_o + (row * p.NP + part) * D + d) = r;
            if (d == 0) {
                // NaN (of a score or a value) outweighs every other partition in the merge, which
                // leaves out partitions without a positive sum: the row is NaN however it is split
                const bool nan = !(den == den) || !(z == z);
                p.part_m[row * p.NP + part] = nan ? 3.4e38f : M;
                p.part_l[row * p.NP + part] = nan ? 1.f : den;
            }
        }
    }
}

template <int D, int BITS, bool FOLD, bool SPARSE, bool SCORED>
cudaError_t launch_decode_int_t(const DecodeParams& p, int G, int q_dtype, cudaStream_t st) {
    constexpr int SMEM = IntCfg<D, BITS, FOLD>::kBytes;
    auto kern = decode_int_kernel<D, BITS, FOLD, SPARSE, SCORED>;
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
    return launch_maybe_pdl(true, kern, dim3(p.NP, p.Hkv, p.S), dim3(IntCfg<D, BITS, FOLD>::kWarps * 32), SMEM, st, p, G,
                            q_dtype == PKV_BF16 ? 1 : 0);
}

template <int BITS, bool SCORED = false>
cudaError_t launch_decode_int(const DecodeParams& p, int G, int q_dtype, cudaStream_t st) {
    const auto run = [&](auto fold) {
        constexpr bool F = decltype(fold)::value;
        if constexpr (SCORED) {
            return p.D == 128 ? launch_decode_int_t<128, BITS, F, false, true>(p, G, q_dtype, st)
                              : launch_decode_int_t<64, BITS, F, false, true>(p, G, q_dtype, st);
        } else {
            if (p.selected)
                return p.D == 128 ? launch_decode_int_t<128, BITS, F, true, false>(p, G, q_dtype, st)
                                  : launch_decode_int_t<64, BITS, F, true, false>(p, G, q_dtype, st);
            return p.D == 128 ? launch_decode_int_t<128, BITS, F, false, false>(p, G, q_dtype, st)
                              : launch_decode_int_t<64, BITS, F, false, false>(p, G, q_dtype, st);
        }
    };
    return G <= 4 ? run(std::true_type{}) : run(std::false_type{});
}

}  // namespace pkv
