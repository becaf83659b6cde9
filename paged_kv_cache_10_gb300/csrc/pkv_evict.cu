// pkv_evict.cu -- eviction from the cache by accumulated attention weight: the
// tokens that each (sequence, KV head) keeps, and their rows moved together.
//
// Selection: of a row's L tokens the first `sink`, the last `recent` and those of
// the largest weights among the others, n in all, ascending.  Weights become
// 32-bit keys that order like them; a radix selection over 11, 11 and 10 bits
// finds the key of the last one kept, exactly, and ties go to the lowest position.
// One CTA a row keeps its keys in shared memory (up to kCachedTokens; a longer row
// reads its weights again in each pass).
//
// Compaction: row kept[i] moves to position i.  kept ascends, so kept[i] >= i: a
// chunk of entries [a, b) writes positions below b and every later entry reads at b
// or above.  So one CTA that takes its entries chunk by chunk, all of a chunk's
// loads before its first store, may write the blocks it reads from, with one
// barrier a chunk.  Columns of a row never meet: they are split over CTAs where
// there are few rows of sequences and heads.
//
// One GB300: the tokens of 8190 for 8 heads chosen in 8.4 us (two dependent loads,
// three passes of barriers: latency), 2048 of them moved in 6.6; those of 32 x 2048 to
// 4096 chosen in 10.2 us, 1000 each moved in 45.3, 0.87 of what a plain copy of as
// many bytes takes.
#include <algorithm>
#include <cstdint>

#include "pkv_int.cuh"

namespace pkv {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kCachedTokens = 40960;  // 160 KB of keys
constexpr int kBins = 2048;

struct SelectTokens {
    const float* weights;
    const int32_t *block_tables, *seq_lens;
    int32_t* kept;
    int32_t MB, NB, Hkv, n, sink, recent, max_len, cached;
    unsigned int* err;
};

// Larger weights have larger keys; -0 equals 0, NaN is below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (!(w == w)) return 0u;
    const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Key of position t of a row that does not fit shared memory.
__device__ __forceinline__ uint32_t load_key(const SelectTokens& p, const int32_t* table, int h, int t) {
    const int blk = load_live(table + t / kBlockSize);
    if (blk < 0 || blk >= p.NB) return 0u;
    return weight_key(load_live(p.weights + (static_cast<int64_t>(blk) * p.Hkv + h) * kBlockSize + t % kBlockSize));
}

// CTA (KV head x, sequence y).
__global__ void __launch_bounds__(kSelThreads) select_tokens_kernel(const SelectTokens p) {
    extern __shared__ uint32_t keys[];  // [p.cached]
    __shared__ uint32_t hists[3][kBins];  // one a pass, all cleared before the first
    __shared__ uint32_t wsum[kSelWarps], wtie[kSelWarps];
    __shared__ uint32_t found_digit, found_left, found_count;
    wait_primary_grid();
    allow_dependent_launch();
    const int h = blockIdx.x, s = blockIdx.y;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int L = load_live(p.seq_lens + s);
    const int cap = min(p.MB * kBlockSize, p.max_len);
    if (L < 0 || L > cap) {
        if (tid == 0 && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
        L = L < 0 ? 0 : cap;
    }
    int32_t* out = p.kept + (static_cast<int64_t>(s) * p.Hkv + h) * p.n;
    if (L <= p.n) {
        for (int i = tid; i < p.n; i += kSelThreads) out[i] = i < L ? i : -1;
        return;
    }
    for (int i = tid; i < p.sink; i += kSelThreads) out[i] = i;
    for (int i = tid; i < p.recent; i += kSelThreads) out[p.n - p.recent + i] = L - p.recent + i;
    const int M = L - p.sink - p.recent;                // tokens to choose from, from position sink on
    const uint32_t k = p.n - p.sink - p.recent;         // as many of them
    if (k == 0) return;
    const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.MB;
    const bool cached = M <= p.cached;
    for (int i = tid; i < 3 * kBins; i += kSelThreads) hists[0][i] = 0u;
    __syncthreads();
    // the keys, four of a block a lane, and with them the first digits' counts
    const int from4 = p.sink & ~3, to = p.sink + M;
#pragma unroll 2
    for (int t = from4 + 4 * tid; t < to; t += 4 * kSelThreads) {
        const int blk = load_live(table + t / kBlockSize);
        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
        const bool ok = blk >= 0 && blk < p.NB;
        if (ok)
            w = load_live(reinterpret_cast<const float4*>(p.weights + (static_cast<int64_t>(blk) * p.Hkv + h) * kBlockSize +
                                                          t % kBlockSize));
        else
            report(p.err, PKV_DEVERR_BLOCK_ID);
        const float v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = t + e - p.sink;
            if (i < 0 || i >= M) continue;
            const uint32_t key = ok ? weight_key(v[e]) : 0u;
            if (cached) keys[i] = key;
            atomicAdd(&hists[0][key >> 21], 1u);
        }
    }
    const auto key_of = [&](int i) { return cached ? keys[i] : load_key(p, table, h, p.sink + i); };

    // keys at or above `from` are kept, and `ties` of those equal to `tie`
    uint32_t prefix = 0u, left = k;
    bool whole = false;  // the last digit's bin is kept in whole
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3 && !whole; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        const int high = shift;  // bits [high, 32) are known
        shift -= bits;
        uint32_t* hist = hists[pass];
        if (pass > 0) {
            for (int i = tid; i < M; i += kSelThreads) {
                const uint32_t key = key_of(i);
                if ((key >> high) == (prefix >> high)) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
            }
        }
        __syncthreads();
        // bins from the top: thread i has the pair 2i, 2i + 1 counted from there
        const uint32_t hi = hist[kBins - 1 - 2 * tid], lo = hist[kBins - 2 - 2 * tid];
        uint32_t sum = hi + lo;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(kAll, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) wsum[warp] = sum;
        __syncthreads();
        uint32_t before = lane < warp ? wsum[lane] : 0u;
        before = __reduce_add_sync(kAll, before);
        const uint32_t end = before + sum, mid = end - lo, begin = mid - hi;  // counts above each bin
        if (begin < left && left <= mid) {
            found_digit = kBins - 1 - 2 * tid;
            found_left = left - begin;
            found_count = hi;
        } else if (mid < left && left <= end) {
            found_digit = kBins - 2 - 2 * tid;
            found_left = left - mid;
            found_count = lo;
        }
        __syncthreads();
        prefix |= found_digit << shift;
        left = found_left;
        whole = found_count == found_left;
    }
    const uint32_t from = whole ? prefix : prefix + 1u;  // keys end at 0xff800000 (+infinity)
    const uint32_t tie = prefix, ties = whole ? 0u : left;

    // ---- ascending output: a warp's positions are consecutive
    const int seg = (M + kSelThreads - 1) / kSelThreads * 32;
    const int i0 = warp * seg, i1 = min(M, i0 + seg);
    uint32_t sel = 0u, eq = 0u;
    for (int i = i0; i < i1; i += 32) {
        const uint32_t key = i + lane < i1 ? key_of(i + lane) : 0u;
        const bool in = i + lane < i1;
        sel += __popc(__ballot_sync(kAll, in && key >= from));
        eq += __popc(__ballot_sync(kAll, in && ties > 0u && key == tie));
    }
    if (lane == 0) {
        wsum[warp] = sel;
        wtie[warp] = eq;
    }
    __syncthreads();
    sel = __reduce_add_sync(kAll, lane < warp ? wsum[lane] : 0u);
    eq = __reduce_add_sync(kAll, lane < warp ? wtie[lane] : 0u);
    for (int i = i0; i < i1; i += 32) {
        const uint32_t key = i + lane < i1 ? key_of(i + lane) : 0u;
        const bool in = i + lane < i1;
        const bool above = in && key >= from, equal = in && ties > 0u && key == tie;
        const uint32_t ba = __ballot_sync(kAll, above), be = __ballot_sync(kAll, equal), below = (1u << lane) - 1u;
        const uint32_t ra = sel + __popc(ba & below), re = eq + __popc(be & below);
        if (above || (equal && re < ties)) out[p.sink + ra + min(re, ties)] = p.sink + i + lane;
        sel += __popc(ba);
        eq += __popc(be);
    }
}

struct Compact {
    const int32_t* kept;
    unsigned char *k_cache, *v_cache;
    float* weights;
    const int32_t *src_tables, *dst_tables, *seq_lens;
    int32_t n, Hkv, NB, src_mb, dst_mb, slices, rows, planes;  // rows: sequences times heads
    unsigned int* err;
};

constexpr int kRowsY = 65535;  // rows of grid axis y; axis z holds the planes of these, of the next ones, ...

// One entry of a list: the bytes from the pool's start to where its row comes from
// and goes to; src < 0: it stays.
struct __align__(16) Move {
    int64_t src, dst;
};

// Moves one head's rows of one pool: 2^lg pieces of type T a row, row(t) + col(u) the
// place of piece u of token t in a tile of tile_bytes, u from u0 on.  The entries of a
// window (one a thread of the CTA) are translated through the tables once, the next window's loads under
// way meanwhile; within it a thread holds PER pieces, and as many of the chunk
// behind them, in registers.  A thread's pieces are all of one column.
template <int THREADS, typename T, int PER, typename Row, typename Col>
__device__ __forceinline__ void move_rows(const Compact& p, Move* win, unsigned char* pool, int64_t tile_bytes, int lg,
                                          int u0, int h, int s, int count, int L, bool rep, Row row, Col col) {
    const int32_t* kept = p.kept + (static_cast<int64_t>(s) * p.Hkv + h) * p.n;
    const int32_t* src_table = p.src_tables + static_cast<int64_t>(s) * p.src_mb;
    const int32_t* dst_table = p.dst_tables + static_cast<int64_t>(s) * p.dst_mb;
    const auto translate = [&](int i) {
        Move m{-1, 0};
        if (i >= count) return m;
        const int b = load_live(dst_table + i / kBlockSize);
        const int t = load_live(kept + i);
        if (t < 0) return m;
        if (t >= L) {
            if (rep) report(p.err, PKV_DEVERR_SEQ_LEN);
            return m;
        }
        const int a = load_live(src_table + t / kBlockSize);
        if (a < 0 || a >= p.NB || b < 0 || b >= p.NB) {
            if (rep) report(p.err, PKV_DEVERR_BLOCK_ID);
            return m;
        }
        if (a == b && t % kBlockSize == i % kBlockSize) return m;  // already there
        m.src = (static_cast<int64_t>(a) * p.Hkv + h) * tile_bytes + row(t % kBlockSize);
        m.dst = (static_cast<int64_t>(b) * p.Hkv + h) * tile_bytes + row(i % kBlockSize);
        return m;
    };
    unsigned char* column = pool + col(u0 + (threadIdx.x & ((1 << lg) - 1)));
    const int first = threadIdx.x >> lg, step = THREADS >> lg;  // this thread's rows of a window
    Move next = translate(threadIdx.x);
    for (int w0 = 0; w0 < count; w0 += THREADS) {
        __syncthreads();  // the window before is through
        win[threadIdx.x] = next;
        __syncthreads();
        next = translate(w0 + THREADS + threadIdx.x);
        const int rows = min(THREADS, count - w0);
        const auto load = [&](int at, T (&x)[PER]) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int i = at + e * step + first;
                const int64_t src = i < rows ? win[i].src : -1;
                if (src >= 0) x[e] = load_live(reinterpret_cast<const T*>(column + src));
            }
        };
        const auto store = [&](int at, const T (&x)[PER]) {
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int i = at + e * step + first;
                if (i < rows) {
                    const Move m = win[i];
                    if (m.src >= 0) *reinterpret_cast<T*>(column + m.dst) = x[e];
                }
            }
        };
        // a chunk's loads before its stores; the loads of chunks behind it read above what it writes
        const int chunk = PER * step;
        T x[PER], y[PER];
        load(0, x);
        for (int at = 0; at < rows; at += 2 * chunk) {
            if (at + chunk < rows) load(at + chunk, y);
            __syncthreads();
            store(at, x);
            if (at + chunk >= rows) break;
            if (at + 2 * chunk < rows) load(at + 2 * chunk, x);
            __syncthreads();
            store(at + chunk, y);
        }
    }
}

// One sequence's and head's part of a plane.
template <int THREADS, int D, int KV>
__device__ __forceinline__ void compact_row(const Compact& p, Move* win, int plane, int s, int h, int count, int L,
                                            bool first) {
    constexpr bool kInt = KV == PKV_INT8 || KV == PKV_INT4;
    const int cut = __ffs(p.slices) - 1;  // log2 of the column slices
    const auto none = [](int) { return 0; };
    const auto one = [&](unsigned char* pool, int64_t tile_bytes, auto type, auto row) {
        using T = decltype(type);
        if (blockIdx.x == 0) move_rows<THREADS, T, 1>(p, win, pool, tile_bytes, 0, 0, h, s, count, L, false, row, none);
    };
    const auto weights = [&] {
        one(reinterpret_cast<unsigned char*>(p.weights), kBlockSize * 4, float{}, [](int t) { return t * 4; });
    };
    if constexpr (!kInt) {
        if (plane == 2) {
            weights();
            return;
        }
        // three pieces a thread and buffer: with four, whose rows lie a power of two apart, 49.2 us
        // against 45.3 for 32 sequences of 1000 tokens; with five 46.1, with two 50.8
        constexpr int ROW = D * (KV == PKV_FP8_E4M3 ? 1 : 2), LG = ROW == 256 ? 4 : (ROW == 128 ? 3 : 2);
        move_rows<THREADS, uint4, 3>(p, win, plane ? p.v_cache : p.k_cache, kBlockSize * ROW, LG - cut,
                                     blockIdx.x << (LG - cut), h, s, count, L, first, [](int t) { return t * ROW; },
                                     [](int u) { return u * 16; });
    } else {
        using L_ = IntTile<D, KV == PKV_INT8 ? 8 : 4>;
        constexpr int LG = L_::RB == 128 ? 3 : (L_::RB == 64 ? 2 : 1);  // 16-byte pieces of a key row
        // both places are a token's plus a byte's
        if (plane == 0) {
            if (blockIdx.x == 0)
                move_rows<THREADS, uint4, 4>(p, win, p.k_cache, L_::kBytes, LG, 0, h, s, count, L, first,
                                             [](int t) { return L_::key(t, 0); }, [](int u) { return L_::key(0, u * 16); });
        } else if (plane == 1) {  // two bytes lie together in a value tile: the codes that are split
            move_rows<THREADS, uint16_t, 8>(p, win, p.v_cache, L_::kBytes, LG + 3 - cut, blockIdx.x << (LG + 3 - cut), h, s,
                                        count, L, false, [](int t) { return L_::val(t, 0); }, [](int u) { return L_::val(0, u * 2); });
        } else if (plane == 4) {
            weights();
        } else {
            one(plane == 3 ? p.v_cache : p.k_cache, L_::kBytes, uint2{}, [](int t) { return L_::param(t); });
        }
    }
}

// CTA (column slice x, sequence and KV head y, plane z) of up to kRowsY rows.  Planes: keys, values, then
// for integer-coded pools their rows' parameters, and the weights last: one pool after
// the other (1000 of 2048 to 4096 tokens, 32 sequences, 8 heads: 45.3 us, 3 less than
// with a head's pools side by side; a copy of as many bytes takes 39.7).
template <int THREADS, int D, int KV>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) compact_kernel(const Compact p) {
    __shared__ Move win[THREADS];
    wait_primary_grid();
    const int plane = blockIdx.z % p.planes, r = static_cast<int>(blockIdx.z / p.planes) * kRowsY + blockIdx.y;
    if (r >= p.rows) return;
    const int s = r / p.Hkv, h = r - s * p.Hkv;
    const bool first = blockIdx.x == 0 && plane == 0;
    int L = load_live(p.seq_lens + s);
    if (L < 0 || L > p.src_mb * kBlockSize) {
        if (threadIdx.x == 0 && first && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
        L = L < 0 ? 0 : p.src_mb * kBlockSize;
    }
    int count = min(p.n, L);
    if (count > p.dst_mb * kBlockSize) {
        if (threadIdx.x == 0 && first && h == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
        count = p.dst_mb * kBlockSize;
    }
    compact_row<THREADS, D, KV>(p, win, plane, s, h, count, L, first);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

pkv_status check_desc(const pkv_cache_desc* d) {
    if (!d || d->num_blocks <= 0 || d->num_kv_heads <= 0 || d->head_size <= 0 || d->block_size <= 0 ||
        !known_kv_dtype(d->kv_dtype))
        return PKV_ERR_INVALID;
    if (d->block_size != kBlockSize || (d->head_size != 64 && d->head_size != 128)) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

template <int THREADS, int D>
void (*compact_of(int kv))(Compact) {
    switch (kv) {
    case PKV_INT8: return compact_kernel<THREADS, D, PKV_INT8>;
    case PKV_INT4: return compact_kernel<THREADS, D, PKV_INT4>;
    case PKV_FP8_E4M3: return compact_kernel<THREADS, D, PKV_FP8_E4M3>;
    default: return compact_kernel<THREADS, D, PKV_BF16>;  // 16-bit rows alike
    }
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_select_tokens(const float* weights, const pkv_cache_desc* d, const int32_t* block_tables,
                                        int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t max_seq_len,
                                        int32_t num_seqs, int32_t num_kept, int32_t sink_tokens, int32_t recent_tokens,
                                        int32_t* kept, void* stream) {
    const pkv_status bad = check_desc(d);
    if (bad != PKV_OK) return bad;
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || max_seq_len < 0 || num_kept <= 0 || sink_tokens < 0 ||
        recent_tokens < 0 || sink_tokens > num_kept || recent_tokens > num_kept - sink_tokens)
        return PKV_ERR_INVALID;
    if (max_blocks_per_seq > 0x7fffffff / kBlockSize || max_seq_len > max_blocks_per_seq * kBlockSize)
        return max_blocks_per_seq > 0x7fffffff / kBlockSize ? PKV_ERR_UNSUPPORTED : PKV_ERR_INVALID;
    if (num_seqs > 65535 || max_seq_len > 0x40000000) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!weights || !block_tables || !seq_lens || !kept || !aligned16(weights) || !aligned4(block_tables) ||
        !aligned4(seq_lens) || !aligned4(kept))
        return PKV_ERR_INVALID;
    SelectTokens p{};
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    p.weights = weights;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.kept = kept;
    p.MB = max_blocks_per_seq;
    p.NB = d->num_blocks;
    p.Hkv = d->num_kv_heads;
    p.n = num_kept;
    p.sink = sink_tokens;
    p.recent = recent_tokens;
    p.max_len = static_cast<int32_t>(std::min<int64_t>((static_cast<int64_t>(max_seq_len) + kBlockSize - 1) / kBlockSize * kBlockSize,
                                                       static_cast<int64_t>(max_blocks_per_seq) * kBlockSize));
    p.cached = std::min(p.max_len, kCachedTokens);
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PKV_ERR_CUDA;
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(select_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCachedTokens * 4) !=
            cudaSuccess)
            return PKV_ERR_CUDA;
        configured[dev] = true;
    }
    const cudaError_t e = launch_maybe_pdl(true, select_tokens_kernel, dim3(p.Hkv, num_seqs), dim3(kSelThreads),
                                           static_cast<size_t>(p.cached) * 4, static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" pkv_status pkv_paged_kv_compact(const int32_t* kept, int32_t num_kept, void* k_cache, void* v_cache,
                                           float* weights, const pkv_cache_desc* d, const int32_t* block_tables,
                                           int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs,
                                           const int32_t* dst_tables, int32_t dst_blocks_per_seq, void* stream) {
    const pkv_status bad = check_desc(d);
    if (bad != PKV_OK) return bad;
    if (num_seqs < 0 || num_kept <= 0 || max_blocks_per_seq <= 0 || dst_blocks_per_seq <= 0) return PKV_ERR_INVALID;
    if (max_blocks_per_seq > 0x7fffffff / kBlockSize || dst_blocks_per_seq > 0x7fffffff / kBlockSize ||
        num_kept > 0x7fffffff - 4096 || num_seqs > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!kept || !k_cache || !v_cache || !block_tables || !seq_lens || !dst_tables || !aligned4(kept) ||
        !aligned4(block_tables) || !aligned4(seq_lens) || !aligned4(dst_tables) || !aligned4(weights) ||
        !aligned16(k_cache) || !aligned16(v_cache))
        return PKV_ERR_INVALID;
    Compact p{};
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    p.kept = kept;
    p.k_cache = static_cast<unsigned char*>(k_cache);
    p.v_cache = static_cast<unsigned char*>(v_cache);
    p.weights = weights;
    p.src_tables = block_tables;
    p.dst_tables = dst_tables;
    p.seq_lens = seq_lens;
    p.n = num_kept;
    p.Hkv = d->num_kv_heads;
    p.NB = d->num_blocks;
    p.src_mb = max_blocks_per_seq;
    p.dst_mb = dst_blocks_per_seq;
    // Columns split over up to four CTAs until there are three an SM (two pools; 45.3
    // against 48.8 us with twice as many for 32 sequences of 1000 tokens).  Where that is
    // not reached by far, what one CTA has under way limits the rate, and CTAs of four
    // times the threads take over (2048 of 8190 tokens, 8 heads: 6.6 us against 11.0).
    if (static_cast<int64_t>(num_seqs) * p.Hkv > int64_t{kRowsY} * (65535 / 5)) return PKV_ERR_UNSUPPORTED;  // grid axis z
    p.rows = num_seqs * p.Hkv;
    const int64_t rows = 2 * static_cast<int64_t>(p.rows);
    p.slices = rows >= 3 * num_sms() ? 1 : (2 * rows >= 3 * num_sms() ? 2 : 4);
    const bool few = rows < num_sms();
    p.planes = (is_int_pool(d->kv_dtype) ? 4 : 2) + (weights ? 1 : 0);
    auto kern = d->head_size == 128 ? (few ? compact_of<1024, 128>(d->kv_dtype) : compact_of<256, 128>(d->kv_dtype))
                                    : (few ? compact_of<1024, 64>(d->kv_dtype) : compact_of<256, 64>(d->kv_dtype));
    const dim3 grid(p.slices, std::min(p.rows, kRowsY), p.planes * ((p.rows + kRowsY - 1) / kRowsY));
    const cudaError_t e = launch_maybe_pdl(true, kern, grid, dim3(few ? 1024 : 256), 0,
                                           static_cast<cudaStream_t>(stream), p);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
