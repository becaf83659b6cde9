// pkv_weights.cu -- each cached token's share of the softmax of a decode step,
// summed over the query heads of its KV head, for eviction by weight.
//
//     w[t] = sum_g 2^(x_g(t) - M_g) / l_g
// from the scores x_g(t) (log2 units) that the scored decode kept and the
// maxima and sums of its partitions.  A head's sum over all its tokens is known
// only when every partition has run, so the share cannot be added up inside
// the decode; keeping a binary32 score for each query head and token costs G / 64
// of a 16-bit cache's bytes at D = 128 and reading the keys again would cost half
// of them.
#include <cstdint>

#include "pkv_decode_impl.cuh"

namespace pkv {
namespace {

constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 512;  // tokens of a CTA

// CTA (tokens [512 x, 512 x + 512), KV head y, sequence z).
template <int G>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const DecodeParams p, const int32_t* new_lens,
                                                                 const int max_len, float* weights) {
    __shared__ float sm_m[G], sm_inv[G];
    wait_primary_grid();
    allow_dependent_launch();
    const int h = blockIdx.y, s = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int L = load_live(p.seq_lens + s);
    const int cap = p.MB * kBlockSize;
    bool bad = L < 0 || L > cap || L > max_len;
    L = L < 0 ? 0 : min(L, min(cap, max_len));
    int fresh = new_lens ? load_live(new_lens + s) : L;
    if (fresh < 0 || fresh > L) {
        bad = true;
        fresh = fresh < 0 ? 0 : L;
    }
    const ScoredRow row = scored_row(p, s, L, bad);
    if (bad && threadIdx.x == 0 && blockIdx.x == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
    const int t0 = blockIdx.x * kWeightTokens;
    if (t0 >= L || t0 + kWeightTokens <= min(row.lo, L - fresh)) return;
    if (warp < G) {  // G <= 8 warps
        const int nparts = row.lo < row.end ? scored_parts(p, row) : 0;
        const int64_t at = (static_cast<int64_t>(s) * p.Hq + h * G + warp) * p.NP;
        float M = kNoScore, den = 0.f;
        for (int i = lane; i < nparts; i += 32) {
            const float l = load_live(p.part_l + at + i);
            if (l > 0.f) {
                const float m = load_live(p.part_m + at + i), n = fmaxf(M, m);
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
    const float* scores = p.scores + (static_cast<int64_t>(s) * p.Hkv + h) * p.span * G;
    const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.MB;
#pragma unroll
    for (int i = 0; i < kWeightTokens / kWeightThreads; ++i) {
        const int t = t0 + i * kWeightThreads + threadIdx.x;
        const bool seen = t >= row.lo && t < row.end, anew = t >= L - fresh;
        if (t >= L || (!seen && !anew)) continue;
        const int phys = load_live(table + t / kBlockSize);
        if (phys < 0 || phys >= p.NB) {
            report(p.err, PKV_DEVERR_BLOCK_ID);
            continue;
        }
        float w = 0.f;
        if (seen) {
            const float* x = scores + static_cast<int64_t>(t - row.start) * G;
#pragma unroll
            for (int g = 0; g < G; ++g) w = fmaf(ex2(load_live(x + g) - sm_m[g]), sm_inv[g], w);
        }
        float* dst = weights + (static_cast<int64_t>(phys) * p.Hkv + h) * kBlockSize + t % kBlockSize;
        *dst = anew ? w : load_live(dst) + w;
    }
}

}  // namespace

cudaError_t launch_weights(const DecodeParams& p, const int32_t* new_lens, int max_seq_len, float* weights,
                           cudaStream_t st) {
    const int max_len = (max_seq_len + kBlockSize - 1) / kBlockSize * kBlockSize;
    if (max_len == 0) return cudaSuccess;
    const dim3 grid((max_len + kWeightTokens - 1) / kWeightTokens, p.Hkv, p.S);
    auto run = [&](auto kern) { return launch_maybe_pdl(true, kern, grid, dim3(kWeightThreads), 0, st, p, new_lens, max_len, weights); };
    switch (p.Hq / p.Hkv) {
    case 1: return run(weights_kernel<1>);
    case 2: return run(weights_kernel<2>);
    case 4: return run(weights_kernel<4>);
    default: return run(weights_kernel<8>);
    }
}

}  // namespace pkv
