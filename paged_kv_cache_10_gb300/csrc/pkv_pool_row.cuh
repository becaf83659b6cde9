// pkv_pool_row.cuh -- eight elements of one cached row as binary32, for every
// pool type, and eight binary32 values as one 16-byte vector of a 16-bit type.
#pragma once

#include <type_traits>

#include "pkv_int.cuh"

namespace pkv {

// Source of eight elements of token t of a tile, as binary32.
template <int D, int KV>
struct PoolRow {
    static constexpr int64_t kTile = KV == PKV_INT8   ? IntTile<D, 8>::kBytes
                                     : KV == PKV_INT4 ? IntTile<D, 4>::kBytes
                                     : KV == PKV_FP8_E4M3 ? kBlockSize * D
                                                          : kBlockSize * D * 2;
    __device__ __forceinline__ static void load(const unsigned char* tile, bool value, int t, int c, float scale,
                                                float* f) {
        if constexpr (KV == PKV_INT8) {
            int_load8<D, 8>(tile, value, t, c, int_params<D, 8>(tile, t), f);
        } else if constexpr (KV == PKV_INT4) {
            int_load8<D, 4>(tile, value, t, c, int_params<D, 4>(tile, t), f);
        } else if constexpr (KV == PKV_FP8_E4M3) {
            const uint2 x = *reinterpret_cast<const uint2*>(tile + t * D + 8 * c);
            const uint32_t w[2] = {x.x, x.y};
            Unpack<E4M3, 8>::run(w, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= scale;
        } else {
            const uint4 x = *reinterpret_cast<const uint4*>(tile + (t * D + 8 * c) * 2);
            if constexpr (KV == PKV_BF16)
                Unpack<BF16, 8>::run(&x.x, f);
            else
                Unpack<F16, 8>::run(&x.x, f);
        }
    }
};

// Eight binary32 values rounded to 16 bits: to nearest ...
template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
    uint4 o;
    uint32_t* w = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, BF16>::value) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
            const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    return o;
}

// ... and outwards, for bounds: down (toward -inf) and up (toward +inf).
template <typename T, bool UP>
__device__ __forceinline__ uint4 pack8_directed(const float* f) {
    uint4 o;
    uint32_t* w = &o.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = f[2 * i + e];
            if constexpr (std::is_same<T, BF16>::value)
                u[e] = __bfloat16_as_ushort(UP ? __float2bfloat16_ru(x) : __float2bfloat16_rd(x));
            else
                u[e] = __half_as_ushort(UP ? __float2half_ru(x) : __float2half_rd(x));
        }
        w[i] = u[0] | (u[1] << 16);
    }
    return o;
}
template <typename T>
__device__ __forceinline__ uint4 pack8_down(const float* f) { return pack8_directed<T, false>(f); }
template <typename T>
__device__ __forceinline__ uint4 pack8_up(const float* f) { return pack8_directed<T, true>(f); }

}  // namespace pkv
