// pkv_weights.cu -- the last part of a scored decode that leaves weights: each
// cached token's share of the softmax, summed over the query heads of its KV
// head, for eviction by weight; and, in the same launch, the merge of the
// decode's partials into the output rows.
//
//     w[t] = sum_g 2^(x_g(t) - M_g) / l_g
// from the scores x_g(t) (log2 units) that the decode kept and the maxima and
// sums of its partitions.  A head's sum over all its tokens is known only when
// every partition has run, so the share cannot be added up inside the decode;
// keeping a binary32 score for each query head and token costs G / 64 of a 16-bit
// cache's bytes at D = 128, and reading the keys again would cost half of them.
//
// A lane takes four tokens of a block: G vectors of scores, one of weights; all
// its loads go out before the heads' sums are known.  The merge has CTAs of its own
// behind those, so that each CTA waits for memory twice: for its row's length, then
// for everything else.
//
// One GB300, bf16: 64 x U[512, 4096] tokens, 32/8 heads 110.0 us with the decode, which
// takes 95.0 without shares (5 of the 15 to write 19 MB of scores, 4 for this launch, 6
// for its loads' latency); 1 x 8190 tokens, 64/8 heads 12.6 against 10.2.
#include <cstdint>

#include "pkv_decode_impl.cuh"

namespace pkv {
namespace {

constexpr int kWeightThreads = 256, kWeightWarps = kWeightThreads / 32;
static_assert(kWeightWarps >= 8, "a warp for each head of a group");
constexpr int kWeightTokens = 4 * kWeightThreads;  // tokens of a CTA
constexpr int kMergeAlone = 8;                     // partitions of a launch up to which a warp merges a row alone

// The log-sum-exp sums of partitions first, first + step, ...: maximum M, sum den relative
// to it and this lane's VD head dimensions of sum_i l_i 2^(m_i - M) o_i; a partition
// without a sum has no output to read.
template <int VD>
__device__ __forceinline__ void add_partials(const float* pm, const float* pl, const float* po, int first, int step,
                                             int nparts, float& M, float& den, float (&acc)[VD]) {
    constexpr int CH = 4;  // partitions whose loads are under way together
    for (int i0 = first; i0 < nparts; i0 += CH * step) {
        float l[CH], m[CH], o[CH][VD], top = M;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = i0 + c * step;
            l[c] = 0.f;
            m[c] = kNoScore;
#pragma unroll
            for (int v = 0; v < VD; ++v) o[c][v] = 0.f;
            if (i >= nparts) continue;
            l[c] = load_live(pl + i);
            m[c] = load_live(pm + i);
            if constexpr (VD == 4) {
                const float4 x = load_live(reinterpret_cast<const float4*>(po + static_cast<int64_t>(i) * 128));
                o[c][0] = x.x; o[c][1] = x.y; o[c][2] = x.z; o[c][3] = x.w;
            } else {
                const float2 x = load_live(reinterpret_cast<const float2*>(po + static_cast<int64_t>(i) * 64));
                o[c][0] = x.x; o[c][1] = x.y;
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) top = l[c] > 0.f ? fmaxf(top, m[c]) : top;
        const float a = ex2(M - top);
        M = top;
        den *= a;
#pragma unroll
        for (int v = 0; v < VD; ++v) acc[v] *= a;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const float w = l[c] > 0.f ? l[c] * ex2(m[c] - top) : 0.f;
            if (w > 0.f) {
                den += w;
#pragma unroll
                for (int v = 0; v < VD; ++v) acc[v] = fmaf(w, o[c][v], acc[v]);
            }
        }
    }
}

// Merge of one head's G output rows (x = 0 .. gridDim of them): a warp a row where a
// launch has few partitions, a CTA a row otherwise.
template <int G, int D, typename QT>
__device__ __forceinline__ void merge_rows(const DecodeParams& p, int x, int h, int s, int nparts) {
    constexpr int VD = D / 32;
    __shared__ float sm_acc[kWeightWarps][D], sm_m[kWeightWarps], sm_l[kWeightWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool alone = p.NP <= kMergeAlone;
    const int g = alone ? warp : x;
    if (g >= G) return;  // a whole warp, or a whole CTA
    const int64_t row = static_cast<int64_t>(s) * p.Hq + h * G + g, at = row * p.NP;
    float acc[VD], M = kNoScore, den = 0.f;
#pragma unroll
    for (int v = 0; v < VD; ++v) acc[v] = 0.f;
    add_partials<VD>(p.part_m + at, p.part_l + at, p.part_o + at * D + lane * VD, alone ? 0 : warp, alone ? 1 : kWeightWarps,
                     nparts, M, den, acc);
    auto* out = reinterpret_cast<typename QT::storage*>(p.out) + row * D;
    if (alone) {
        const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
        for (int v = 0; v < VD; ++v) out[lane * VD + v] = from_float<QT>(acc[v] * inv);
        return;
    }
#pragma unroll
    for (int v = 0; v < VD; ++v) sm_acc[warp][lane * VD + v] = acc[v];
    if (lane == 0) {
        sm_m[warp] = M;
        sm_l[warp] = den;
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float top = kNoScore, sum = 0.f, r = 0.f;
#pragma unroll
        for (int w = 0; w < kWeightWarps; ++w) top = fmaxf(top, sm_m[w]);
#pragma unroll
        for (int w = 0; w < kWeightWarps; ++w) {
            const float c = ex2(sm_m[w] - top);
            sum = fmaf(c, sm_l[w], sum);
            r = fmaf(c, sm_acc[w][threadIdx.x], r);
        }
        out[threadIdx.x] = from_float<QT>(sum > 0.f ? r / sum : 0.f);
    }
}

// CTA (tokens [1024 x, 1024 x + 1024), KV head y, sequence z), and behind the
// tokens' CTAs those of the merge.
template <int G, int D, typename QT>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const DecodeParams p, const int32_t* new_lens,
                                                                 const int max_len, float* weights) {
    __shared__ float sm_m[G], sm_inv[G];
    wait_primary_grid();
    allow_dependent_launch();
    const int h = blockIdx.y, s = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the decode's row, and the part of it that weights cover
    const int given = load_live(p.seq_lens + s);
    int fresh = new_lens ? load_live(new_lens + s) : 0x7fffffff;
    const int cap = p.MB * kBlockSize;
    bool bad = given < 0 || given > cap;
    const ScoredRow row = scored_row(p, s, given < 0 ? 0 : min(given, cap), bad);
    const int nparts = row.lo < row.end ? scored_parts(p, row) : 0;
    const int tiles = (max_len + kWeightTokens - 1) / kWeightTokens;
    if (static_cast<int>(blockIdx.x) >= tiles) {
        merge_rows<G, D, QT>(p, blockIdx.x - tiles, h, s, nparts);
        return;
    }
    bad |= given > max_len;
    const int L = given < 0 ? 0 : min(given, min(cap, max_len));
    if (!new_lens) fresh = L;
    if (fresh < 0 || fresh > L) {
        bad = true;
        fresh = fresh < 0 ? 0 : L;
    }
    if (bad && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
    const int t0 = blockIdx.x * kWeightTokens;
    if (t0 >= L || t0 + kWeightTokens <= min(row.lo, L - fresh)) return;

    // ---- this lane's four tokens
    const int t = t0 + 4 * threadIdx.x;
    float x[4][G] = {};
    float4 old = make_float4(0.f, 0.f, 0.f, 0.f);
    float* dst = nullptr;
    if (t < L && t + 4 > min(row.lo, L - fresh)) {
        const int phys = load_live(p.block_tables + static_cast<int64_t>(s) * p.MB + t / kBlockSize);
        if (phys < 0 || phys >= p.NB) {
            report(p.err, PKV_DEVERR_BLOCK_ID);
        } else {
            dst = weights + (static_cast<int64_t>(phys) * p.Hkv + h) * kBlockSize + t % kBlockSize;
            if (t < L - fresh) old = load_live(reinterpret_cast<const float4*>(dst));
        }
        // a block in front of the row's first has no scores; the scores of a block that lies
        // behind its last token are not read
        if (t >= row.start && t < row.end) {
            const float4* src = reinterpret_cast<const float4*>(
                p.scores + ((static_cast<int64_t>(s) * p.Hkv + h) * p.span + (t - row.start)) * G);
            float4 v[G];
#pragma unroll
            for (int i = 0; i < G; ++i) v[i] = load_live(src + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int at = e * G + g;
                    const float4 q = v[at / 4];
                    x[e][g] = at % 4 == 0 ? q.x : (at % 4 == 1 ? q.y : (at % 4 == 2 ? q.z : q.w));
                }
        }
    }

    // ---- each head's maximum and the reciprocal of its sum
    if (warp < G) {
        const int64_t at = (static_cast<int64_t>(s) * p.Hq + h * G + warp) * p.NP;
        float M = kNoScore, den = 0.f;
        for (int i = lane; i < nparts; i += 32) {
            const float l = load_live(p.part_l + at + i), m = load_live(p.part_m + at + i);
            if (l > 0.f) {
                const float n = fmaxf(M, m);
                den = den * ex2(M - n) + l * ex2(m - n);
                M = n;
            }
        }
#pragma unroll
        for (int mask = 16; mask > 0; mask >>= 1) {
            const float m = __shfl_xor_sync(kFull, M, mask), d = __shfl_xor_sync(kFull, den, mask), n = fmaxf(M, m);
            den = den * ex2(M - n) + d * ex2(m - n);
            M = n;
        }
        if (lane == 0) {
            sm_m[warp] = M;
            sm_inv[warp] = den > 0.f ? 1.f / den : 0.f;
        }
    }
    __syncthreads();

    if (dst) {
        float w[4];
        bool put[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool seen = t + e >= row.lo && t + e < row.end && t + e < L, anew = t + e >= L - fresh;
            float sum = 0.f;
#pragma unroll
            for (int g = 0; g < G; ++g) sum = fmaf(ex2(x[e][g] - sm_m[g]), sm_inv[g], sum);
            const float before = e == 0 ? old.x : (e == 1 ? old.y : (e == 2 ? old.z : old.w));
            w[e] = (anew ? 0.f : before) + (seen ? sum : 0.f);
            put[e] = t + e < L && (seen || anew);
        }
        if (put[0] && put[1] && put[2] && put[3]) {
            *reinterpret_cast<float4*>(dst) = make_float4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (put[e]) dst[e] = w[e];
        }
    }
}

template <int D, typename QT>
cudaError_t launch_weights_t(const DecodeParams& p, const int32_t* new_lens, int max_len, float* weights,
                             cudaStream_t st) {
    const int merge = p.NP <= kMergeAlone ? 1 : p.Hq / p.Hkv;
    const dim3 grid((max_len + kWeightTokens - 1) / kWeightTokens + merge, p.Hkv, p.S);
    auto run = [&](auto kern) {
        return launch_maybe_pdl(true, kern, grid, dim3(kWeightThreads), 0, st, p, new_lens, max_len, weights);
    };
    switch (p.Hq / p.Hkv) {
    case 1: return run(weights_kernel<1, D, QT>);
    case 2: return run(weights_kernel<2, D, QT>);
    case 4: return run(weights_kernel<4, D, QT>);
    default: return run(weights_kernel<8, D, QT>);
    }
}

}  // namespace

cudaError_t launch_weights(const DecodeParams& p, const int32_t* new_lens, int max_seq_len, int q_dtype, float* weights,
                           cudaStream_t st) {
    const int max_len = (max_seq_len + kBlockSize - 1) / kBlockSize * kBlockSize;
    if (q_dtype == PKV_BF16)
        return p.D == 128 ? launch_weights_t<128, BF16>(p, new_lens, max_len, weights, st)
                          : launch_weights_t<64, BF16>(p, new_lens, max_len, weights, st);
    return p.D == 128 ? launch_weights_t<128, F16>(p, new_lens, max_len, weights, st)
                      : launch_weights_t<64, F16>(p, new_lens, max_len, weights, st);
}

}  // namespace pkv
