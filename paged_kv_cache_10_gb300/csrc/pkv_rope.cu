// pkv_rope.cu -- rotary positions: a step's queries and keys rotated by their
// positions and its keys and values written to their slots, in one pass.
//
// Pair i of a head's first R elements turns by the angle 2 pi pos f_i, f_i in
// turns a position:  (a, b) -> m (a cos - b sin, b cos + a sin).
//
// The angle.  pos f_i in binary32 would be off by 2^-24 of a number of turns
// that reaches 10^5 at far positions.  Here f_i = hi + lo is a pair of binary32
// and pos a sum of a multiple of 4096 and a rest, both exact in binary32; each
// product's rounding error is taken exactly by a fused multiply-add, whole
// turns are dropped from products and errors before they are added up, and
// sincospi takes the rest: within 2^-23 of a turn (plus pos 2^-51), a fifth of
// a binary32 step of an angle of one radian, at no table of positions.
//
// The pass is bound by HBM: q is read and written once, k and v read once
// and written once in the pool's type.  A lane holds 16 elements of a row whose
// pairs are complete in it (half layout: two 8-element vectors R / 2 apart;
// interleaved: 16 elements in a row), so nothing but a coded row's extrema crosses
// lanes.  A CTA's tokens share their cosines and sines through shared memory, one
// sincospi for each pair and token.
//
// One GB300, 128 elements rotated of 128: 8192 tokens, 32/8 heads, bf16 31.9 us, 0.93
// of the measured copy bandwidth on 201 MB; 64 tokens 2.0 us, a launch's latency.
#include <cstdint>

#include "pkv_append.cuh"
#include "pkv_pool_row.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 128;

struct RopeParams {
    const unsigned char *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, o_stride;  // bytes from a token's row to the next one's
    unsigned char* q_out;
    const int32_t* positions;
    const int64_t* slots;
    const float2* freqs;  // [R / 2] (hi, lo), turns a position
    unsigned char *k_cache, *v_cache;
    int64_t num_slots;
    int32_t T, Hq, Hkv, R, interleaved;
    int32_t tokens;  // of a CTA
    int32_t items;   // 16-element items of a token
    int32_t share;   // items of a token that a CTA takes
    float magnitude, k_scale, v_scale;
    unsigned int* err;
};

// m (cos, sin) of 2 pi pos (hi + lo).
__device__ __forceinline__ float2 rotation(int pos, float2 f, float m) {
    const float a = static_cast<float>(pos & ~4095), b = static_cast<float>(pos & 4095);
    const float pa = __fmul_rn(a, f.x), pb = __fmul_rn(b, f.x);
    const float ea = __fmaf_rn(a, f.x, -pa), eb = __fmaf_rn(b, f.x, -pb);  // exact
    const float la = __fmul_rn(a, f.y), lb = __fmul_rn(b, f.y);
    const auto part = [](float x) { return __fsub_rn(x, rintf(x)); };  // exact
    const float turns = part(part(pa) + part(pb)) + (part(ea) + part(la) + (eb + lb));
    float s, c;
    sincospif(2.f * turns, &s, &c);
    return make_float2(c * m, s * m);
}

// Eight rotated pairs: x, y the 8-element vectors of an item, cs its (cos, sin, cos, sin) quads.
template <typename IT>
__device__ __forceinline__ void rotate16(uint4& x, uint4& y, const float4 (&cs)[4], bool interleaved) {
    float a[8], b[8];
    Unpack<IT, 8>::run(&x.x, a);
    Unpack<IT, 8>::run(&y.x, b);
    const auto turn = [](float& u, float& v, float c, float s) {
        const float t = fmaf(u, c, -__fmul_rn(v, s));
        v = fmaf(v, c, __fmul_rn(u, s));
        u = t;
    };
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn(a[2 * i], a[2 * i + 1], i & 1 ? cs[i / 2].z : cs[i / 2].x, i & 1 ? cs[i / 2].w : cs[i / 2].y);
            turn(b[2 * i], b[2 * i + 1], i & 1 ? cs[2 + i / 2].z : cs[2 + i / 2].x, i & 1 ? cs[2 + i / 2].w : cs[2 + i / 2].y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn(a[2 * i], b[2 * i], cs[i].x, cs[i].y);
            turn(a[2 * i + 1], b[2 * i + 1], cs[i].z, cs[i].w);
        }
    }
    x = pack8<IT>(a);
    y = pack8<IT>(b);
}

// CTA (token group x, share y of a token's items).
template <int D, int KV, typename IT>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeParams p) {
    constexpr int LPR = D / 16;  // lanes of a row
    constexpr bool kInt = KV == PKV_INT8 || KV == PKV_INT4;
    constexpr int UNROLL = 3;
    extern __shared__ float4 sm_cs[];  // [token][quad 0 .. 3][item of the rotated part]
    wait_primary_grid();  // a programmatic dependent of the kernel before it on the stream
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
    const int first = blockIdx.y * p.share, per = min(p.share, p.items - first);
    const int total = nt * per;
    const int NR = p.R / 16;  // rotated items of a row

    // Items in rounds of UNROLL a lane: their loads go out before the angles are
    // ready (first round) or the items before them are written.  The rounds are the
    // same for a CTA's lanes, since a coded row's shuffles need all of them.
    for (int base = 0; base < total; base += UNROLL * kRopeThreads) {
        uint4 x[UNROLL][2];
        int tok[UNROLL], hs[UNROLL], va[UNROLL], vb[UNROLL], cc[UNROLL];
        int64_t slot[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int i = base + u * kRopeThreads + tid;
            x[u][0] = x[u][1] = make_uint4(0u, 0u, 0u, 0u);
            slot[u] = -1;
            hs[u] = -1;
            tok[u] = cc[u] = va[u] = vb[u] = 0;
            if (i >= total) continue;
            const int j = i / per, it = first + i - j * per;
            const int h = it / LPR, c = it % LPR;
            const int64_t t = t0 + j;
            tok[u] = j;
            hs[u] = h;
            cc[u] = c;
            if (h >= p.Hq + p.Hkv) {  // a value row
                va[u] = c;
                vb[u] = c + LPR;
            } else if (c >= NR) {
                va[u] = 2 * c;
                vb[u] = 2 * c + 1;
            } else {
                va[u] = p.interleaved ? 2 * c : c;
                vb[u] = p.interleaved ? 2 * c + 1 : c + NR;
            }
            const unsigned char* row = h < p.Hq           ? p.q + t * p.q_stride + static_cast<int64_t>(h) * (D * 2)
                                       : h < p.Hq + p.Hkv ? p.k + t * p.k_stride + static_cast<int64_t>(h - p.Hq) * (D * 2)
                                                          : p.v + t * p.v_stride + static_cast<int64_t>(h - p.Hq - p.Hkv) * (D * 2);
            x[u][0] = load_live(reinterpret_cast<const uint4*>(row) + va[u]);
            x[u][1] = load_live(reinterpret_cast<const uint4*>(row) + vb[u]);
            if (h >= p.Hq) {
                slot[u] = load_live(p.slots + t);
                if (slot[u] >= p.num_slots) {
                    if (h == p.Hq && c == 0) report(p.err, PKV_DEVERR_SLOT);
                    slot[u] = -1;
                }
            }
        }
        if (base == 0) {
            for (int i = tid; i < nt * (p.R / 2); i += kRopeThreads) {
                const int j = i / (p.R / 2), pair = i - j * (p.R / 2);
                const float2 cs = rotation(load_live(p.positions + t0 + j), load_live(p.freqs + pair), p.magnitude);
                const int c = pair / 8, e = pair % 8;
                reinterpret_cast<float2*>(sm_cs)[((j * 4 + e / 2) * NR + c) * 2 + e % 2] = cs;
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const bool value = hs[u] >= p.Hq + p.Hkv;
            if (hs[u] >= 0 && !value && cc[u] < NR) {
                float4 cs[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) cs[k] = sm_cs[(tok[u] * 4 + k) * NR + cc[u]];
                rotate16<IT>(x[u][0], x[u][1], cs, p.interleaved != 0);
            }
            if (hs[u] >= 0 && hs[u] < p.Hq) {
                uint4* o = reinterpret_cast<uint4*>(p.q_out + (t0 + tok[u]) * p.o_stride + static_cast<int64_t>(hs[u]) * (D * 2));
                o[va[u]] = x[u][0];
                o[vb[u]] = x[u][1];
            }
            if constexpr (kInt) {
                uint32_t w[2][2];
                float2 sz = make_float2(0.f, 0.f);
                // some lane of the warp holds part of a row to be coded
                if (__any_sync(0xffffffffu, slot[u] >= 0)) sz = int_encode16<D, KV == PKV_INT8 ? 8 : 4, IT>(x[u], w);
                if (slot[u] >= 0) {
                    using L = IntTile<D, KV == PKV_INT8 ? 8 : 4>;
                    const int head = value ? hs[u] - p.Hq - p.Hkv : hs[u] - p.Hq, t = static_cast<int>(slot[u]) & 15;
                    unsigned char* tile = (value ? p.v_cache : p.k_cache) + ((slot[u] >> 4) * p.Hkv + head) * L::kBytes;
                    int_store8<D, L::kBits>(tile, value, t, va[u], w[0]);
                    int_store8<D, L::kBits>(tile, value, t, vb[u], w[1]);
                    if (cc[u] == 0) *reinterpret_cast<float2*>(tile + L::param(t)) = sz;
                }
            } else if (slot[u] >= 0) {
                const int head = value ? hs[u] - p.Hq - p.Hkv : hs[u] - p.Hq;
                const int64_t row = ((slot[u] >> 4) * p.Hkv + head) * kBlockSize + (slot[u] & 15);
                unsigned char* pool = value ? p.v_cache : p.k_cache;
                if constexpr (KV == PKV_FP8_E4M3) {
                    const float sc = value ? p.v_scale : p.k_scale;
                    uint2* o = reinterpret_cast<uint2*>(pool + row * D);
                    o[va[u]] = encode_e4m3x8<IT>(x[u][0], sc);
                    o[vb[u]] = encode_e4m3x8<IT>(x[u][1], sc);
                } else {
                    uint4* o = reinterpret_cast<uint4*>(pool + row * (D * 2));
                    o[va[u]] = x[u][0];
                    o[vb[u]] = x[u][1];
                }
            }
        }
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int D, typename IT>
cudaError_t launch_rope(const RopeParams& p, int kv_dtype, dim3 grid, cudaStream_t st) {
    void (*kern)(RopeParams) = nullptr;
    switch (kv_dtype) {
    case PKV_F16: kern = rope_append_kernel<D, PKV_F16, F16>; break;
    case PKV_BF16: kern = rope_append_kernel<D, PKV_BF16, BF16>; break;
    case PKV_FP8_E4M3: kern = rope_append_kernel<D, PKV_FP8_E4M3, IT>; break;
    case PKV_INT8: kern = rope_append_kernel<D, PKV_INT8, IT>; break;
    default: kern = rope_append_kernel<D, PKV_INT4, IT>; break;
    }
    return launch_maybe_pdl(true, kern, grid, dim3(kRopeThreads), static_cast<size_t>(p.tokens) * (p.R / 2) * 8, st, p);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_paged_rope_append(const void* q, int64_t q_stride, int32_t num_q_heads, const void* k,
                                            int64_t k_stride, const void* v, int64_t v_stride, int32_t in_dtype,
                                            int32_t num_tokens, const int32_t* positions, const int64_t* slot_mapping,
                                            const float* freqs, int32_t rotary_dim, int32_t interleaved,
                                            float magnitude, void* k_cache, void* v_cache, const pkv_cache_desc* d,
                                            void* q_out, int64_t q_out_stride, void* stream) {
    if (!d || num_tokens < 0 || num_q_heads < 0 || d->num_blocks <= 0 || d->num_kv_heads <= 0 || d->head_size <= 0 ||
        d->block_size <= 0 || !known_kv_dtype(d->kv_dtype))
        return PKV_ERR_INVALID;
    if (d->kv_dtype == PKV_FP8_E4M3 && !(d->k_scale > 0.f && d->v_scale > 0.f)) return PKV_ERR_INVALID;
    if (in_dtype != PKV_F16 && in_dtype != PKV_BF16) return PKV_ERR_INVALID;
    if (d->block_size != kBlockSize || (d->head_size != 64 && d->head_size != 128)) return PKV_ERR_UNSUPPORTED;
    if ((d->kv_dtype == PKV_F16 || d->kv_dtype == PKV_BF16) && in_dtype != d->kv_dtype) return PKV_ERR_UNSUPPORTED;
    if (!(magnitude > -3.0e38f && magnitude < 3.0e38f)) return PKV_ERR_INVALID;
    const int64_t D = d->head_size;
    if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16) return PKV_ERR_INVALID;
    if (num_tokens == 0) return PKV_OK;
    const int64_t heads = static_cast<int64_t>(num_q_heads) + 2 * static_cast<int64_t>(d->num_kv_heads);
    const auto bad_stride = [&](int64_t s, int64_t h) { return s % 8 != 0 || (num_tokens > 1 && s < h * D); };
    if (bad_stride(k_stride, d->num_kv_heads) || bad_stride(v_stride, d->num_kv_heads)) return PKV_ERR_INVALID;
    if (num_q_heads > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out) || bad_stride(q_stride, num_q_heads) ||
                            bad_stride(q_out_stride, num_q_heads)))
        return PKV_ERR_INVALID;
    if (!k || !v || !positions || !slot_mapping || !freqs || !k_cache || !v_cache) return PKV_ERR_INVALID;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
        (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) ||
        (reinterpret_cast<uintptr_t>(freqs) & 7u))
        return PKV_ERR_INVALID;
    if (heads * (D / 16) > 0xffff * kRopeThreads) return PKV_ERR_UNSUPPORTED;  // a token's items: one grid axis
    unsigned int* err = error_word();
    if (!err) return PKV_ERR_CUDA;
    RopeParams p{};
    p.q = static_cast<const unsigned char*>(q);
    p.k = static_cast<const unsigned char*>(k);
    p.v = static_cast<const unsigned char*>(v);
    p.q_stride = 2 * q_stride;
    p.k_stride = 2 * k_stride;
    p.v_stride = 2 * v_stride;
    p.o_stride = 2 * q_out_stride;
    p.q_out = static_cast<unsigned char*>(q_out);
    p.positions = positions;
    p.slots = slot_mapping;
    p.freqs = reinterpret_cast<const float2*>(freqs);
    p.k_cache = static_cast<unsigned char*>(k_cache);
    p.v_cache = static_cast<unsigned char*>(v_cache);
    p.num_slots = static_cast<int64_t>(d->num_blocks) * kBlockSize;
    p.T = num_tokens;
    p.Hq = num_q_heads;
    p.Hkv = d->num_kv_heads;
    p.R = rotary_dim;
    p.interleaved = interleaved != 0;
    p.items = static_cast<int32_t>(heads * (D / 16));
    p.magnitude = magnitude;
    p.k_scale = d->k_scale;
    p.v_scale = d->v_scale;
    p.err = err;
    // Few tokens: a token's items spread over CTAs, one a lane, for the shortest chain.
    // Many: two tokens a CTA, whose angles cost it one sincospi a lane (8192 tokens, 32/8
    // heads: 31.9 us; four tokens 33.7, eight 36.0).
    const bool few = num_tokens <= 4 * num_sms();
    p.tokens = few ? 1 : 2;
    p.share = few ? kRopeThreads : p.items;
    const dim3 grid((num_tokens + p.tokens - 1) / p.tokens, (p.items + p.share - 1) / p.share);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (D == 128)
        e = in_dtype == PKV_BF16 ? launch_rope<128, BF16>(p, d->kv_dtype, grid, st) : launch_rope<128, F16>(p, d->kv_dtype, grid, st);
    else
        e = in_dtype == PKV_BF16 ? launch_rope<64, BF16>(p, d->kv_dtype, grid, st) : launch_rope<64, F16>(p, d->kv_dtype, grid, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
