// pkv_int.cuh -- integer-coded KV pools (PKV_INT8, PKV_INT4): the tile layout
// and the row codec shared by the append, read, staging, key-bounds and
// decode kernels.
//
// A row (one token of one KV head) of D values x is held as unsigned codes of
// b bits with a binary32 scale and zero taken from the row itself:
//   lo = min x, hi = max x, scale = (hi - lo) / (2^b - 1), zero = lo,
//   code = min(rint((x - lo) * (1 / scale)), 2^b - 1),  value = zero + scale * code
// each step one IEEE binary32 operation, so that the codes are the same on
// every machine.  A scale below 2^-126 (a constant row) is stored as 0.  A row with
// a NaN, or whose hi - lo is not finite, is held as codes 0 with scale and zero NaN,
// so that it reads back as NaN instead of as numbers that it did not hold.
//
// A tile (16 tokens of one block and KV head, in one pool) is 16 * RB code
// bytes (RB = D * b / 8) followed by 16 pairs (scale, zero), one contiguous
// run of 640 to 2176 bytes, a multiple of 128: one 1-D bulk copy brings codes
// and parameters together, and a block copy or swap moves both without
// knowing about them.  The code bytes are permuted so that the tensor-core
// decode reads its MMA fragments from a tile as it lies, free of
// shared-memory bank conflicts and without a byte shuffle:
//   keys    byte k of token t: panel k / 64 of [16 tokens][min(RB, 64)] bytes
//   values  byte k of token t is byte x = (k / 2) * 4 + (t % 2) * 2 + k % 2 of
//           token pair t / 2: panel x / 32 of [8 pairs][32] bytes
// (a 32-bit word of a value pair holds two bytes of the even token and the
// same two of the odd one, so masking it gives f16 pairs along the tokens,
// the contraction axis of P V).
#pragma once

#include <type_traits>

#include "pkv_device.cuh"

namespace pkv {

template <int D, int BITS>
struct IntTile {
    static_assert((D == 64 || D == 128) && (BITS == 4 || BITS == 8), "");
    static constexpr int RB = D * BITS / 8;            // code bytes of a row
    static constexpr int KW = RB < 64 ? RB : 64;       // bytes of a key panel's row
    static constexpr int kCodes = kBlockSize * RB;     // code bytes of a tile
    static constexpr int kBytes = kCodes + kBlockSize * 8;
    static constexpr int kD = D, kBits = BITS;
    static_assert(kBytes % 128 == 0, "shared-memory stages keep their bank alignment");
    __host__ __device__ static constexpr int key(int t, int k) { return (k / 64) * (16 * KW) + t * KW + k % 64; }
    __host__ __device__ static constexpr int val(int t, int k) {
        const int x = (k / 2) * 4 + (t % 2) * 2 + k % 2;
        return (x / 32) * 256 + (t / 2) * 32 + x % 32;
    }
    __host__ __device__ static constexpr int param(int t) { return kCodes + t * 8; }
};

// The values of a word's four bytes: a byte under the exponent of 2^23 is that
// float plus the code, exactly, which spares the integer conversion.
__device__ __forceinline__ void int_value4(uint32_t w, float2 sz, float* f, int step) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        f[i * step] = fmaf(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | i)) - 8388608.f, sz.x, sz.y);
}

// Eight elements 8 * c .. 8 * c + 7 of token t of a tile in global memory, with the
// row's (scale, zero) sz.
template <int D, int BITS>
__device__ __forceinline__ float2 int_params(const unsigned char* tile, int t) {
    return *reinterpret_cast<const float2*>(tile + IntTile<D, BITS>::param(t));
}
template <int D, int BITS>
__device__ __forceinline__ void int_load8(const unsigned char* tile, bool value, int t, int c, float2 sz, float* f) {
    using L = IntTile<D, BITS>;
    uint32_t w[BITS / 4];  // the 8 elements' code bytes, in order
    if (!value) {
        const unsigned char* p = tile + L::key(t, c * BITS);
        if constexpr (BITS == 8) {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            w[0] = x.x;
            w[1] = x.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        }
    } else {
        const unsigned char* p = tile + L::val(t, c * BITS);
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) {
            const uint32_t a = *reinterpret_cast<const uint16_t*>(p + 8 * i);
            const uint32_t b = *reinterpret_cast<const uint16_t*>(p + 8 * i + 4);
            w[i] = a | (b << 16);
        }
    }
    if constexpr (BITS == 4) {
        int_value4(w[0] & 0x0f0f0f0fu, sz, f, 2);
        int_value4((w[0] >> 4) & 0x0f0f0f0fu, sz, f + 1, 2);
    } else {
        int_value4(w[0], sz, f, 1);
        int_value4(w[1], sz, f + 4, 1);
    }
}

// x / (2^BITS - 1), correctly rounded, for x >= 0: with y the correctly rounded
// reciprocal of the divisor, q = rn(x y) is within an ulp, the remainder r = x -
// q (2^BITS - 1) is exact in a fused multiply-add, and rn(q + r y) is the rounded
// quotient (Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Outside the range where no step can
// underflow or overflow, the division itself.
template <int BITS>
__device__ __forceinline__ float div_const(float x) {
    constexpr float d = BITS == 8 ? 255.f : 15.f;
    constexpr float y = 1.f / d;
    if (!(x > 0x1p-90f && x < 0x1p120f)) return __fdiv_rn(x, d);
    const float q = __fmul_rn(x, y);
    return __fmaf_rn(__fmaf_rn(-q, d, x), y, q);
}

// A row held by D / 16 consecutive lanes, two 16-byte vectors of eight 16-bit
// elements each, to code bytes: w[i] receives those of vector i, in order; (scale,
// zero) is the row's.  Every lane of the warp takes part in the shuffles.  The
// extrema are found on 16-bit pairs, (min, -max) in one register from the first
// shuffle on.
template <int D, int BITS, typename IT>
__device__ __forceinline__ float2 int_encode16(const uint4 (&x)[2], uint32_t (&w)[2][2]) {
    using P2 = typename std::conditional<std::is_same<IT, BF16>::value, __nv_bfloat162, __half2>::type;
    const uint32_t xw[2][4] = {{x[0].x, x[0].y, x[0].z, x[0].w}, {x[1].x, x[1].y, x[1].z, x[1].w}};
    const P2* v = reinterpret_cast<const P2*>(&xw[0][0]);
    P2 mn = v[0], mx = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        mn = __hmin2_nan(mn, v[i]);
        mx = __hmax2_nan(mx, v[i]);
    }
    P2 key;
    key.x = __hmin_nan(mn.x, mn.y);
    key.y = __hneg(__hmax_nan(mx.x, mx.y));
#pragma unroll
    for (int m = 1; m < D / 16; m <<= 1) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&key), m);
        key = __hmin2_nan(key, *reinterpret_cast<const P2*>(&o));
    }
    const float lo = to_float(key.x), hi = -to_float(key.y), range = __fsub_rn(hi, lo);
    const bool finite = range < INFINITY;  // false for NaN
    float scale = div_const<BITS>(range);
    if (!(scale >= 0x1p-126f)) scale = 0.f;
    const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
    // rint by adding 2^23 (round to nearest, ties to even, like rint): the code is
    // the sum's low bits.  (x - lo) * inv <= top (1 + 2^-22), so no code passes top.
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float f[8];
        Unpack<IT, 8>::run(xw[r], f);
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            c[e] = __float_as_uint(__fadd_rn(__fmul_rn(__fsub_rn(f[e], lo), inv), 8388608.f));
        if constexpr (BITS == 8) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[r][i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040),
                                      __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = c[2 * i] + (c[2 * i + 1] << 4);  // low byte: both codes
            w[r][0] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        }
        if (!finite) w[r][0] = w[r][1] = 0u;
    }
    return finite ? make_float2(scale, lo) : make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
}

// Stores the code bytes of elements 8c .. 8c + 7.
template <int D, int BITS>
__device__ __forceinline__ void int_store8(unsigned char* tile, bool value, int t, int c, const uint32_t* w) {
    using L = IntTile<D, BITS>;
    if (!value) {
        unsigned char* p = tile + L::key(t, c * BITS);
        if constexpr (BITS == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
        unsigned char* p = tile + L::val(t, c * BITS);
#pragma unroll
        for (int i = 0; i < BITS / 4; ++i) {
            *reinterpret_cast<uint16_t*>(p + 8 * i) = static_cast<uint16_t>(w[i]);
            *reinterpret_cast<uint16_t*>(p + 8 * i + 4) = static_cast<uint16_t>(w[i] >> 16);
        }
    }
}

// Calls fn(IntTile<D, BITS>) for an integer pool type and head size.
template <typename Fn>
inline cudaError_t with_int_tile(int kv_dtype, int D, Fn&& fn) {
    if (kv_dtype == PKV_INT8) return D == 128 ? fn(IntTile<128, 8>{}) : fn(IntTile<64, 8>{});
    return D == 128 ? fn(IntTile<128, 4>{}) : fn(IntTile<64, 4>{});
}

}  // namespace pkv
