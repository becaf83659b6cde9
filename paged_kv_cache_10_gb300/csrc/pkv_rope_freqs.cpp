// pkv_rope_freqs.cpp -- the frequencies of rotary positions, in 64 bits on the
// host: turns per position of every rotated pair, scaled for long contexts,
// each as a pair of binary32 whose sum holds 48 bits of it.
#include <cmath>
#include <cstdint>

#include "../../include/pagedkv.h"

extern "C" pkv_status pkv_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                                           int32_t original_len, double low, double high, float* freqs) {
    if (rotary_dim <= 0 || rotary_dim % 2 || !freqs || !(base > 1.0) || !std::isfinite(base)) return PKV_ERR_INVALID;
    if (scaling < PKV_ROPE_NONE || scaling > PKV_ROPE_PARTS) return PKV_ERR_INVALID;
    if (scaling != PKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return PKV_ERR_INVALID;
    if (scaling == PKV_ROPE_NTK && rotary_dim < 4) return PKV_ERR_INVALID;
    if (scaling == PKV_ROPE_PARTS && (original_len <= 0 || !(low < high) || !std::isfinite(low) || !std::isfinite(high)))
        return PKV_ERR_INVALID;
    const double two_pi = 6.283185307179586476925286766559;
    const double R = rotary_dim;
    const double b = scaling == PKV_ROPE_NTK ? base * std::pow(factor, R / (R - 2.0)) : base;
    for (int32_t i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(b, -2.0 * i / R);  // radians a position
        if (scaling == PKV_ROPE_LINEAR) f /= factor;
        if (scaling == PKV_ROPE_PARTS) {
            const double turns = original_len * f / two_pi;  // over the original context
            const double g = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
            f = (1.0 - g) * f / factor + g * f;
        }
        const double turns = f / two_pi;
        const float hi = static_cast<float>(turns);
        freqs[2 * i] = hi;
        freqs[2 * i + 1] = static_cast<float>(turns - static_cast<double>(hi));
    }
    return PKV_OK;
}
