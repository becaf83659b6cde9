// pkv_int_cache.cu -- quantising a cache as it is written, and reading it back:
// the append into integer-coded pools, the read of cached rows by slot (every
// pool type), and the 16-bit copy of integer-coded blocks that prefill reads.
//
// All three are bound by HBM: they move 16-byte vectors of 16-bit values on
// one side and a lane's 4 to 8 code bytes on the other.  D / 16 consecutive
// lanes hold a row, two vectors of eight elements each (vectors c and c + D / 16, so
// that a row's loads and stores stay contiguous over its lanes), so a row's
// minimum and maximum are 2 or 3 shuffle steps and no shared memory is used.
//
// Measured on one GB300: 8192 tokens x 8 heads x 128 at 4 bits written in 10.3 us
// and read back in 9.8, 18.4 together, 0.61 of the measured copy bandwidth on 75.8
// MB (11.2 us); at 8 bits 26.5 and 14.3 (7.6 each).  Neither fills a unit (append,
// cold: 32 % of DRAM, 64 % of the issue slots; read: 10 %, 54 %): a group of lanes
// has one row in flight an iteration and waits for its loads.  At 8 bits the append
// waits for its stores too, value codes two bytes at a time: 2.5 M sector writes
// for 0.56 M sectors of codes.  One round of eight resident CTAs an SM, four a pool,
// beats a row's share a CTA (18.7 against 19.8 us), sixteen elements a lane beat
// eight (22.2 us).  The 64 tokens of a decode step are latency: 1.6 to 2.7 us a launch.
#include <cstdint>

#include "pkv_append.cuh"
#include "pkv_pool_row.cuh"

namespace pkv {
namespace {

// Quotient of a row number below 2^31 by the number of KV heads, as a product.
struct RowDiv {
    uint32_t mul, d;
    int shift;
};
RowDiv row_div(int d) {
    int s = 0;
    while ((1ll << s) < d) ++s;
    return {static_cast<uint32_t>((1ull << (31 + s)) / d + 1), static_cast<uint32_t>(d), 31 + s};
}
__device__ __forceinline__ uint32_t quotient(uint32_t n, RowDiv v) {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * v.mul) >> v.shift);
}

// Append into an integer-coded pool: one group of D / 16 lanes per row (t, h),
// blockIdx.y = 0 keys, 1 values.  Lanes of a warp whose row is padding or out
// of range still take part in the group's shuffles.  Eight CTAs an SM, four a pool,
// leave a thread 32 registers.
template <int D, int BITS, typename IT>
__global__ void __launch_bounds__(256, 8) append_int_kernel(const uint4* k, const uint4* v,
                                                         const int64_t* slots, unsigned char* kc,
                                                         unsigned char* vc, uint32_t rows, RowDiv heads,
                                                         int64_t num_slots, unsigned int* err) {
    using L = IntTile<D, BITS>;
    constexpr int LPR = D / 16, RPC = 256 / LPR;  // lanes of a row, rows of a CTA
    wait_primary_grid();  // a programmatic dependent of the kernel before it on the stream
    const bool value = blockIdx.y != 0;
    const uint4* src = value ? v : k;
    unsigned char* pool = value ? vc : kc;
    const int c = threadIdx.x % LPR;
    // rows < 2^31 and gridDim.x * RPC < 2^20: no overflow.  The loop's end is the same
    // for a CTA's lanes, since the shuffles need all of them.
    for (uint32_t base = blockIdx.x * RPC; base < rows; base += gridDim.x * RPC) {
        const uint32_t row = base + threadIdx.x / LPR;
        int64_t slot = -1;
        uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        uint32_t h = 0;
        if (row < rows) {
            const uint32_t t = quotient(row, heads);
            h = row - t * heads.d;
            const uint4* p = src + static_cast<int64_t>(row) * (2 * LPR) + c;
            x[0] = load_live(p);
            x[1] = load_live(p + LPR);
            slot = load_live(slots + t);
            if (slot >= num_slots) {
                if (h == 0 && c == 0 && !value) report(err, PKV_DEVERR_SLOT);
                slot = -1;
            }
        }
        uint32_t w[2][2];
        const float2 sz = int_encode16<D, BITS, IT>(x, w);
        if (slot >= 0) {
            // tiles of a pool count below 2^32
            unsigned char* tile =
                pool + static_cast<uint64_t>(static_cast<uint32_t>(slot >> 4) * heads.d + h) * L::kBytes;
            const int t = static_cast<int>(slot) & 15;
            int_store8<D, BITS>(tile, value, t, c, w[0]);
            int_store8<D, BITS>(tile, value, t, c + LPR, w[1]);
            if (c == 0) *reinterpret_cast<float2*>(tile + L::param(t)) = sz;
        }
    }
}

// Read by slot: D / 16 lanes per row (t, h), blockIdx.y = 0 keys, 1 values.
template <int D, int KV, typename OT>
__global__ void __launch_bounds__(256) read_kernel(const unsigned char* kc,
                                                   const unsigned char* vc,
                                                   const int64_t* slots, uint4* k_out, uint4* v_out,
                                                   uint32_t rows, RowDiv heads, int64_t num_slots, float k_scale,
                                                   float v_scale, unsigned int* err) {
    constexpr int LPR = D / 16, RPC = 256 / LPR;
    wait_primary_grid();
    const bool value = blockIdx.y != 0;
    const unsigned char* pool = value ? vc : kc;
    uint4* out = value ? v_out : k_out;
    const float scale = value ? v_scale : k_scale;
    const int c = threadIdx.x % LPR;
    for (uint32_t row = blockIdx.x * RPC + threadIdx.x / LPR; row < rows; row += gridDim.x * RPC) {
        const uint32_t t = quotient(row, heads), h = row - t * heads.d;
        const int64_t slot = load_live(slots + t);
        if (slot < 0) continue;
        if (slot >= num_slots) {
            if (h == 0 && c == 0 && !value) report(err, PKV_DEVERR_SLOT);
            continue;
        }
        const uint32_t tile = static_cast<uint32_t>(slot >> 4) * heads.d + h;  // below 2^32
        const unsigned char* p = pool + tile * PoolRow<D, KV>::kTile;
        float f[2][8];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            PoolRow<D, KV>::load(p, value, static_cast<int>(slot) & 15, c + i * LPR, scale, f[i]);
        uint4* o = out + static_cast<int64_t>(row) * (2 * LPR) + c;
        o[0] = pack8<OT>(f[0]);
        o[LPR] = pack8<OT>(f[1]);
    }
}

// 16-bit copy of integer-coded blocks for prefill: one CTA per (logical block
// j, sequence s, pool z).  A block id outside the pool is reported and its copy
// zeroed, so that the attention pass reads no stale bytes.
template <int D, int BITS, typename OT>
__global__ void __launch_bounds__(256) stage_int_kernel(const unsigned char* __restrict__ kc,
                                                        const unsigned char* __restrict__ vc,
                                                        const int32_t* __restrict__ block_tables,
                                                        const int32_t* __restrict__ seq_lens, int MB, int NB, int Hkv,
                                                        uint4* __restrict__ k_copy, uint4* __restrict__ v_copy,
                                                        int32_t* __restrict__ table_copy, unsigned int* err) {
    using L = IntTile<D, BITS>;
    allow_dependent_launch();  // the attention kernel may start its setup
    const int j = blockIdx.x, s = blockIdx.y;
    const bool value = blockIdx.z != 0;
    const int len = __ldg(seq_lens + s);  // the attention pass reports a bad length
    const int nblk = len <= 0 ? 0 : min((len - 1) / kBlockSize + 1, MB);
    if (j >= nblk) return;
    const int64_t at = static_cast<int64_t>(s) * MB + j;
    const int id = __ldg(block_tables + at);
    const bool bad = id < 0 || id >= NB;
    if (threadIdx.x == 0 && !value) {
        table_copy[at] = static_cast<int32_t>(at);
        if (bad) report(err, PKV_DEVERR_BLOCK_ID);
    }
    // rows past the sequence's end may never have been written: the copy holds zeros there
    const int valid = min(kBlockSize, len - j * kBlockSize);
    const int per_head = kBlockSize * D / 8, total = Hkv * per_head;
    const unsigned char* src = (value ? vc : kc) + (bad ? 0 : static_cast<int64_t>(id) * Hkv * L::kBytes);
    uint4* dst = (value ? v_copy : k_copy) + at * total;
    for (int i = threadIdx.x; i < total; i += 256) {
        const int h = i / per_head, t = i % per_head / (D / 8), c = i % (D / 8);
        float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (!bad && t < valid) {
            const unsigned char* tile = src + static_cast<int64_t>(h) * L::kBytes;
            int_load8<D, BITS>(tile, value, t, c, int_params<D, BITS>(tile, t), f);
        }
        dst[i] = pack8<OT>(f);
    }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

unsigned row_grid(int64_t rows, int rows_per_cta) {
    const int64_t need = (rows + rows_per_cta - 1) / rows_per_cta, cap = static_cast<int64_t>(num_sms()) * 4;
    return static_cast<unsigned>(need < cap ? need : cap);
}

template <int D, typename OT>
cudaError_t launch_read(int kv, const void* kc, const void* vc, const int64_t* slots, void* ko, void* vo, int64_t rows,
                        const pkv_cache_desc* d, unsigned int* err, cudaStream_t st) {
    void (*kern)(const unsigned char*, const unsigned char*, const int64_t*, uint4*, uint4*, uint32_t, RowDiv, int64_t,
                 float, float, unsigned int*) = nullptr;
    switch (kv) {
    case PKV_F16: kern = read_kernel<D, PKV_F16, F16>; break;
    case PKV_BF16: kern = read_kernel<D, PKV_BF16, BF16>; break;
    case PKV_FP8_E4M3: kern = read_kernel<D, PKV_FP8_E4M3, OT>; break;
    case PKV_INT8: kern = read_kernel<D, PKV_INT8, OT>; break;
    default: kern = read_kernel<D, PKV_INT4, OT>; break;
    }
    return launch_maybe_pdl(true, kern, dim3(row_grid(rows, 256 * 16 / D), 2), dim3(256), 0, st,
                            static_cast<const unsigned char*>(kc), static_cast<const unsigned char*>(vc), slots,
                            static_cast<uint4*>(ko), static_cast<uint4*>(vo), static_cast<uint32_t>(rows),
                            row_div(d->num_kv_heads), static_cast<int64_t>(d->num_blocks) * kBlockSize, d->k_scale,
                            d->v_scale, err);
}

}  // namespace

cudaError_t launch_append_int(const void* k, const void* v, int in_dtype, int64_t num_tokens, const int64_t* slots,
                              void* k_cache, void* v_cache, const pkv_cache_desc* d, unsigned int* err,
                              cudaStream_t st) {
    return with_int_tile(d->kv_dtype, d->head_size, [&](auto tile) {
        using L = decltype(tile);
        constexpr int D = L::kD, BITS = L::kBits;
        const int64_t rows = num_tokens * d->num_kv_heads;
        auto kern = in_dtype == PKV_BF16 ? append_int_kernel<D, BITS, BF16> : append_int_kernel<D, BITS, F16>;
        return launch_maybe_pdl(true, kern, dim3(row_grid(rows, 256 * 16 / D), 2), dim3(256), 0, st,
                                static_cast<const uint4*>(k), static_cast<const uint4*>(v), slots,
                                static_cast<unsigned char*>(k_cache), static_cast<unsigned char*>(v_cache),
                                static_cast<uint32_t>(rows), row_div(d->num_kv_heads),
                                static_cast<int64_t>(d->num_blocks) * kBlockSize, err);
    });
}

cudaError_t launch_stage_int(int kv_dtype, int D, int q_dtype, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* seq_lens, int S, int MB, int NB, int Hkv,
                             void* k_copy, void* v_copy, int32_t* table_copy, unsigned int* err, cudaStream_t st) {
    return with_int_tile(kv_dtype, D, [&](auto tile) {
        using L = decltype(tile);
        constexpr int HD = L::kD, BITS = L::kBits;
        auto kern = q_dtype == PKV_BF16 ? stage_int_kernel<HD, BITS, BF16> : stage_int_kernel<HD, BITS, F16>;
        kern<<<dim3(static_cast<unsigned>(MB), static_cast<unsigned>(S), 2), 256, 0, st>>>(
            static_cast<const unsigned char*>(k_cache), static_cast<const unsigned char*>(v_cache), block_tables,
            seq_lens, MB, NB, Hkv, static_cast<uint4*>(k_copy), static_cast<uint4*>(v_copy), table_copy, err);
        return cudaGetLastError();
    });
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_cache_block_bytes(const pkv_cache_desc* d) {
    if (!d || d->num_kv_heads <= 0 || !known_kv_dtype(d->kv_dtype) || d->block_size != kBlockSize ||
        (d->head_size != 64 && d->head_size != 128))
        return 0;
    return static_cast<size_t>(d->num_kv_heads * tile_bytes(d->kv_dtype, d->head_size));
}

extern "C" pkv_status pkv_paged_kv_read(const int64_t* slot_mapping, int32_t num_tokens, const void* k_cache,
                                        const void* v_cache, const pkv_cache_desc* d, void* k_out, void* v_out,
                                        int32_t out_dtype, void* stream) {
    if (!d || num_tokens < 0 || d->num_blocks <= 0 || d->num_kv_heads <= 0 || d->head_size <= 0 || d->block_size <= 0)
        return PKV_ERR_INVALID;
    if (!known_kv_dtype(d->kv_dtype) || (out_dtype != PKV_F16 && out_dtype != PKV_BF16)) return PKV_ERR_INVALID;
    if (d->kv_dtype == PKV_FP8_E4M3 && !(d->k_scale > 0.f && d->v_scale > 0.f)) return PKV_ERR_INVALID;
    if (d->block_size != kBlockSize || (d->head_size != 64 && d->head_size != 128)) return PKV_ERR_UNSUPPORTED;
    if ((d->kv_dtype == PKV_F16 || d->kv_dtype == PKV_BF16) && out_dtype != d->kv_dtype) return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!slot_mapping || !k_cache || !v_cache || !k_out || !v_out) return PKV_ERR_INVALID;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID;
    unsigned int* err = error_word();
    if (!err) return PKV_ERR_CUDA;
    const int64_t rows = static_cast<int64_t>(num_tokens) * d->num_kv_heads;
    if (rows > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (d->head_size == 128)
        e = out_dtype == PKV_BF16
                ? launch_read<128, BF16>(d->kv_dtype, k_cache, v_cache, slot_mapping, k_out, v_out, rows, d, err, st)
                : launch_read<128, F16>(d->kv_dtype, k_cache, v_cache, slot_mapping, k_out, v_out, rows, d, err, st);
    else
        e = out_dtype == PKV_BF16
                ? launch_read<64, BF16>(d->kv_dtype, k_cache, v_cache, slot_mapping, k_out, v_out, rows, d, err, st)
                : launch_read<64, F16>(d->kv_dtype, k_cache, v_cache, slot_mapping, k_out, v_out, rows, d, err, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
