// pkv_score.cuh -- what scored attention does to a score, shared by the decode
// kernels, their merge and the prefill.
//
//     x = scale * q.k;  x = cap * tanh(x / cap);  x = x - slope * |p - t|
// for the query at position p and the key at position t, in log2 units: the
// kernels take y = q.k * qk_scale with qk_scale = scale / cap (or scale *
// log2(e) without a cap), cap_out = cap * log2(e) and slopes times log2(e).
#pragma once

#include "pkv_device.cuh"

namespace pkv {

// 2^x with the hardware approximation (relative error ~2^-22; -inf -> 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / x with the hardware approximation (one unit in the last place).
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kNoScore = -3e38f;  // softmax reference before the first score
constexpr float kLog2e = 1.4426950408889634f;

// tanh within 2^-22 of 1, and within 2^-22 of itself below 1/4: 1 - 2 / (e^2|y| + 1),
// which cancels for small |y|, or there the first five terms of the Taylor
// series (the sixth is 2^-26.8 of y at 1/4).
__device__ __forceinline__ float tanh_score(float y) {
    const float a = fabsf(y), y2 = y * y;
    const float big = copysignf(fmaf(-2.f, rcp(ex2(a * (2.f * kLog2e)) + 1.f), 1.f), y);
    const float c = fmaf(y2, fmaf(y2, fmaf(y2, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
    const float small = fmaf(y * y2, c, y);
    return a < 0.25f ? small : big;
}

// Scored decode: the first token a row of L tokens attends to, through its
// window and its first position (L where nothing is left).
__device__ __forceinline__ int scored_first(int window, const int32_t* first, int s, int L) {
    int lo = first ? load_live(first + s) : 0;
    if (window > 0 && lo < L - window) lo = L - window;
    return lo < 0 ? 0 : (lo > L ? L : lo);
}

// A row's tokens [lo, end) and the first one of the block that lo lies in.
struct ScoredRow {
    int lo, start, end;
};

// The row of sequence s with L tokens; a row longer than the launch was sized
// for (bad is set) loses its last ones.
__device__ __forceinline__ ScoredRow scored_row(const DecodeParams& p, int s, int L, bool& bad) {
    ScoredRow r;
    r.lo = scored_first(p.window, p.first, s, L);
    r.start = r.lo / kBlockSize * kBlockSize;
    r.end = L;
    if (L - r.start > p.span) {
        bad = true;
        r.end = r.start + p.span;
    }
    return r;
}

// Partitions of the row; one for a row with nothing in it (its CTA writes the
// zeros) unless the merge writes every row.
__device__ __forceinline__ int scored_parts(const DecodeParams& p, const ScoredRow& r) {
    if (r.lo >= r.end) return p.cascade ? 0 : 1;
    return (r.end - r.start + p.P - 1) / p.P;
}

__device__ __forceinline__ float scored_slope(const DecodeParams& p, int head) {
    return p.slopes ? load_live(p.slopes + head) * kLog2e : 0.f;
}

// The score at distance dist >= 0 from y = q.k * qk_scale.
__device__ __forceinline__ float scored(const DecodeParams& p, float y, float slope, int dist) {
    const float x = p.cap_out > 0.f ? p.cap_out * tanh_score(y) : y;
    return fmaf(-slope, static_cast<float>(dist), x);
}

}  // namespace pkv
