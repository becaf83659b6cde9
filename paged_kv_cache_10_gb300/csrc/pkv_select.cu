// pkv_select.cu -- block selection for sparse decode: the channelwise key bounds
// of every block, the blocks whose bounds promise the highest scores, and the
// entry point of the attention over them.
//
// For a block with key bounds lo_d <= k_td <= hi_d no token of it can score
// above  u_g = sum_d max(q_gd lo_d, q_gd hi_d)  for query head g.  A block's
// score is max_g u_g over the G query heads of a KV head, and a row (sequence,
// KV head) keeps the blocks of the highest scores.  With q+ = max(q, 0) and
// q- = min(q, 0), u_g = q+_g . hi + q-_g . lo: one product of length 2 D with the
// block's bounds as they are stored, on the warp-level tensor-core MMA with 16
// blocks on its M rows and the G heads on its N columns.
#include <algorithm>
#include <cstdint>

#include "pkv_decode_mma.cuh"
#include "pkv_int.cuh"
#include "pkv_pool_row.cuh"

namespace pkv {
namespace {

// ------------------------------------------------------------- key bounds
// One CTA per (block in reach of the new tokens, sequence): a thread takes
// eight channels of one KV head and reads them of the block's (at most 16)
// tokens, 16 independent loads in flight; lanes of a row read it whole, so
// no reduction across threads is needed.  Bound by the chain length -> table ->
// keys -> bounds: 2.6 us for the 256 blocks of a decode step (5.6 MB), 4.1 us for
// 8 x 1024 new tokens (19 MB, 4.6 TB/s).
template <int D, int KV, typename OT>
__global__ void __launch_bounds__(128) key_bounds_kernel(const unsigned char* kc,
                                                         const int32_t* block_tables, int MB,
                                                         const int32_t* seq_lens,
                                                         const int32_t* new_lens, int max_new, int NB,
                                                         int Hkv, float k_scale, unsigned char* bounds,
                                                         unsigned int* err) {
    wait_primary_grid();  // a programmatic dependent of the kernel before it on the stream
    const int s = blockIdx.y;
    const int len = load_live(seq_lens + s);
    const int fresh = new_lens ? load_live(new_lens + s) : len;
    if (len < 0 || len > MB * kBlockSize || fresh < 0 || fresh > len || fresh > max_new) {
        if (threadIdx.x == 0 && blockIdx.x == 0) report(err, PKV_DEVERR_SEQ_LEN);
        return;
    }
    if (fresh == 0) return;
    const int j = (len - fresh) / kBlockSize + blockIdx.x;
    if (j > (len - 1) / kBlockSize) return;
    const int id = load_live(block_tables + static_cast<int64_t>(s) * MB + j);
    if (id < 0 || id >= NB) {
        if (threadIdx.x == 0) report(err, PKV_DEVERR_BLOCK_ID);
        return;
    }
    const int valid = min(kBlockSize, len - j * kBlockSize);
    for (int i = threadIdx.x; i < Hkv * (D / 8); i += blockDim.x) {
        const int h = i / (D / 8), c = i % (D / 8);
        const int64_t at = static_cast<int64_t>(id) * Hkv + h;
        const unsigned char* tile = kc + at * PoolRow<D, KV>::kTile;
        float lo[8], hi[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo[e] = INFINITY;
            hi[e] = -INFINITY;
        }
        // past the last token the last one again: the loads need no branch between
        // them, and an extremum does not mind
#pragma unroll
        for (int t = 0; t < kBlockSize; ++t) {
            float f[8];
            PoolRow<D, KV>::load(tile, false, min(t, valid - 1), c, k_scale, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                lo[e] = fminf(lo[e], f[e]);
                hi[e] = fmaxf(hi[e], f[e]);
            }
        }
        unsigned char* out = bounds + (at * 2 * D + 8 * c) * 2;
        *reinterpret_cast<uint4*>(out) = pack8_down<OT>(lo);
        *reinterpret_cast<uint4*>(out + D * 2) = pack8_up<OT>(hi);
    }
}

// ----------------------------------------------------------------- scores
struct SelectParams {
    const void* q;
    const unsigned char* bounds;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    int32_t* selected;
    float* score;   // [S * Hkv][cols]
    float* top;     // [S * Hkv][cols / 16]  largest |bound| of 16 blocks
    double* exact;  // [S * Hkv][cols]  64-bit scores of the blocks near the border
    int S, Hq, Hkv, G, MB, NB, cols, n, sink, recent;
    int tiles;      // 16-block tiles one warp of the score kernel takes
    int smem_cols;  // columns of a row that the selection keeps in shared memory
    unsigned int* err;
};

// The row's blocks, clamped to what the launch covers.
__device__ __forceinline__ int row_blocks(const SelectParams& p, int s, bool& bad) {
    int len = load_live(p.seq_lens + s);
    const int cap = min(p.MB, p.cols);
    bad = len < 0 || (len > 0 && (len - 1) / kBlockSize >= cap);
    return len <= 0 ? 0 : min((len - 1) / kBlockSize + 1, cap);
}

// Largest |x| of packed 16-bit pairs (NaN passed over).
template <typename T>
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t x) {
    using P2 = typename std::conditional<std::is_same<T, BF16>::value, __nv_bfloat162, __half2>::type;
    const P2 r = __hmax2(*reinterpret_cast<const P2*>(&m), __habs2(*reinterpret_cast<const P2*>(&x)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Shared memory of the score kernel: a ring of 16-block tiles per warp.  A
// block's 2 D bound elements lie at a pitch of 64 bytes modulo 128, so that the
// eight lanes of a 16-byte read phase (two rows, four chunks) hit all banks.
template <int D>
struct ScoreCfg {
    static constexpr int kWarps = 4;
    static constexpr int kStages = 2;
    static constexpr int kCtasPerSm = D == 128 ? 3 : 5;
    static constexpr int kRow = 4 * D;  // bytes of a block's bounds for one KV head
    static constexpr int kPitch = kRow + 64;
    static constexpr int kStage = 16 * kPitch;
    static constexpr int kBarOffset = kWarps * kStages * kStage;
    static constexpr int kMaskOffset = kBarOffset + kWarps * kStages * 8;
    static constexpr int kBytes = kMaskOffset + kWarps * kStages * 4 + 128;
    static_assert(kPitch % 128 == 64 && kCtasPerSm * (kBytes + 1024) <= 228 * 1024, "residency");
};

// One warp per (KV head, run of p.tiles 16-block tiles, sequence).  A tile's 16
// rows come by one bulk copy each, issued by 16 lanes, kStages tiles ahead, with
// the ids of the next tiles already in registers.  Lane (g8, qd) reads
// 16-byte chunks qd, qd + 4, ... of rows g8 and g8 + 8 as MMA fragments, which
// only permutes the contraction axis; Q's fragments follow the same order.
//
// Bound by HBM: 32 x 30000 .. 32768 tokens, 8 KV heads, 259 MB of bounds in 40.3
// us, 0.95 of the measured copy bandwidth.  Fragments loaded straight from global
// memory took 85 us (14 warps an SM with one tile in flight each), 16-byte
// asynchronous copies instead of bulk ones 3 to 5 us more.
template <int D, typename T>
__global__ void __launch_bounds__(128) block_score_kernel(const SelectParams p) {
    using C = ScoreCfg<D>;
    constexpr bool kBF = std::is_same<T, BF16>::value;
    constexpr int CH = D / 16;  // 16-byte chunks of a row per lane
    constexpr int NST = C::kStages;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((128 - (smem_addr(smem_raw) & 127)) & 127);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, qd = lane & 3;
    const int64_t unit = blockIdx.x * 4ll + warp;
    const int h = static_cast<int>(unit % p.Hkv), s = blockIdx.y;
    const int first = static_cast<int>(unit / p.Hkv) * p.tiles;
    unsigned char* ring = smem + warp * NST * C::kStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOffset) + warp * NST;
    volatile uint32_t* masks = reinterpret_cast<uint32_t*>(smem + C::kMaskOffset) + warp * NST;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < NST; ++i) mbar_init(&bars[i], 1);
        mbar_init_fence();
    }
    // A programmatic dependent of the kernel before it on the stream.  Its own, the
    // selection, reads q and the lengths and writes short rows before it waits, so
    // it may start only now.
    wait_primary_grid();
    allow_dependent_launch();
    bool bad;
    const int nblk = row_blocks(p, s, bad);
    if (bad && unit == 0 && lane == 0) report(p.err, PKV_DEVERR_SEQ_LEN);
    if (first * 16 >= nblk || nblk <= p.n) return;  // a row that keeps every block needs no scores
    const int tiles = min(p.tiles, (nblk + 15) / 16 - first);

    __syncwarp();
    const uint64_t pol = policy_evict_first();
    const int32_t* table = p.block_tables + static_cast<int64_t>(s) * p.MB;
    // Lane l of `ids` number k & 1 holds the id of block l of tile pair k (-1 for
    // none); a pair is loaded two pairs ahead of its use.
    const auto ids_of = [&](int k) {
        const int j = (first + 2 * k) * 16 + lane;
        return 2 * k + (lane >> 4) < tiles && j < nblk ? load_live(table + j) : -1;
    };
    int ids[2] = {ids_of(0), ids_of(1)};
    const auto issue = [&](int t, int stage) {  // warp-uniform; tiles in order
        const int src = (lane & 15) + 16 * (t & 1);
        const int id0 = __shfl_sync(kFull, ids[0], src), id1 = __shfl_sync(kFull, ids[1], src);
        const int id = lane < 16 ? ((t >> 1) & 1 ? id1 : id0) : -1;
        const bool in = id >= 0 && id < p.NB;
        if (!in && lane < 16 && (first + t) * 16 + lane < nblk && h == 0) report(p.err, PKV_DEVERR_BLOCK_ID);
        const uint32_t mask = __ballot_sync(kFull, in);
        if (lane == 0) {
            masks[stage] = mask;
            mbar_arrive_expect_tx(&bars[stage], __popc(mask) * C::kRow);
        }
        __syncwarp();
        if (in)
            bulk_g2s(ring + stage * C::kStage + lane * C::kPitch,
                     p.bounds + (id * static_cast<int64_t>(p.Hkv) + h) * C::kRow, C::kRow, &bars[stage], pol);
        if (t & 1) {
            if ((t >> 1) & 1)
                ids[1] = ids_of((t >> 1) + 2);
            else
                ids[0] = ids_of((t >> 1) + 2);
        }
    };
    int issued = 0;
#pragma unroll
    for (int i = 0; i < NST; ++i)
        if (issued < tiles) {
            issue(issued, i);
            ++issued;
        }
    // ---- Q's fragments: elements of [q-, q+] of head g8
    uint32_t qb[2 * CH][2];
    {
        const bool live = g8 < p.G;
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.q) +
                                                          (static_cast<int64_t>(s) * p.Hq + h * p.G + (live ? g8 : 0)) * D * 2);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = 4 * j + qd;  // chunk of the 2 D row: the first D / 8 are lo's
            const bool low = c < D / 8;
            const uint4 x = live ? load_live(row + (low ? c : c - D / 8)) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // keep the elements whose sign bit says q < 0 (lo) or q >= 0 (hi)
                const uint32_t neg = ((w[i] >> 15) & 0x00010001u) * 0xffffu;
                y[i] = w[i] & (low ? neg : ~neg);
            }
            qb[2 * j][0] = y[0];
            qb[2 * j][1] = y[1];
            qb[2 * j + 1][0] = y[2];
            qb[2 * j + 1][1] = y[3];
        }
    }
    const int64_t out = (static_cast<int64_t>(s) * p.Hkv + h) * p.cols + static_cast<int64_t>(first) * 16;
    bool aborted = false;
    uint32_t phase = 0;
    for (int t0 = 0; t0 < tiles && !aborted; t0 += NST) {
#pragma unroll
        for (int st = 0; st < NST; ++st) {
            const int t = t0 + st;
            if (t >= tiles) break;
            if (!mbar_wait(&bars[st], phase)) {
                if (lane == 0) report(p.err, PKV_DEVERR_TIMEOUT);
                aborted = true;
                break;
            }
            const uint32_t mask = masks[st];
            const uint32_t base = smem_addr(ring + st * C::kStage) + g8 * C::kPitch + qd * 16;
            float sa[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            uint32_t big0 = 0u, big1 = 0u;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const uint4 a = lds128(base + 64 * j), b = lds128(base + 8 * C::kPitch + 64 * j);
                mma16816a<kBF>(sa[0], a.x, b.x, a.y, b.y, qb[2 * j][0], qb[2 * j][1]);
                mma16816a<kBF>(sa[1], a.z, b.z, a.w, b.w, qb[2 * j + 1][0], qb[2 * j + 1][1]);
                big0 = abs_max2<T>(abs_max2<T>(abs_max2<T>(abs_max2<T>(big0, a.x), a.y), a.z), a.w);
                big1 = abs_max2<T>(abs_max2<T>(abs_max2<T>(abs_max2<T>(big1, b.x), b.y), b.z), b.w);
            }
            const bool ok[2] = {(mask >> g8 & 1u) != 0u, (mask >> (g8 + 8) & 1u) != 0u};
            const uint32_t big = abs_max2<T>(ok[0] ? big0 : 0u, ok[1] ? big1 : 0u);
            float v[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float x = sa[0][2 * r] + sa[1][2 * r], y = sa[0][2 * r + 1] + sa[1][2 * r + 1];
                float m = -INFINITY;  // NaN scores are dropped: such a block ranks last
                if (2 * qd < p.G) m = fmaxf(m, x);
                if (2 * qd + 1 < p.G) m = fmaxf(m, y);
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
                m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
                v[r] = ok[r] ? m : -INFINITY;  // a row without a block holds stale bytes
            }
            if (qd == 0) {
                p.score[out + t * 16 + g8] = v[0];
                p.score[out + t * 16 + g8 + 8] = v[1];
            }
            const uint32_t top = __reduce_max_sync(kFull, max(big >> 16, big & 0xffffu));
            if (lane == 0) {
                const uint16_t b = static_cast<uint16_t>(top);
                p.top[out / 16 + t] = to_float(*reinterpret_cast<const typename T::storage*>(&b));
            }
            __syncwarp();
            if (issued < tiles) {
                issue(issued, st);
                ++issued;
            }
        }
        phase ^= 1u;
    }
    if (aborted) {  // no copy may outlive the CTA
        for (int k = 0; k < NST; ++k) {
            const int t = issued - 1 - k;
            if (t < 0) break;
            (void)mbar_wait(&bars[t % NST], (t / NST) & 1);
        }
    }
}

// -------------------------------------------------------------- selection
constexpr int kSelThreads = 256;
constexpr int kSmemCols = 16384;  // 64 KiB of a row's scores; longer rows stay in the workspace
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 1024;
constexpr int kSelNear = 256;  // blocks near the border that are ranked pair by pair

// Exclusive sum of v over the CTA's threads in order.
__device__ __forceinline__ int cta_scan(int v, int* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int y = __shfl_up_sync(kFull, x, m);
        if (lane >= m) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) before += red[w];
    return before + x - v;
}

// Bits that order like the double they come from.
__device__ __forceinline__ uint64_t order64(double x) {
    const int64_t b = __double_as_longlong(x);
    return static_cast<uint64_t>(b) ^ (b < 0 ? ~0ull : 1ull << 63);
}

// This lane's D / 32 channels of a block's bounds for KV head h, as binary32;
// false for a negative j or a block id outside the pool.
template <int D, typename T>
__device__ __forceinline__ bool lane_bounds(const SelectParams& p, int s, int h, int j, float* lo, float* hi) {
    constexpr int V = D / 32;
    const int id = j >= 0 ? load_live(p.block_tables + static_cast<int64_t>(s) * p.MB + j) : -1;
    const bool ok = id >= 0 && id < p.NB;
    const unsigned char* b =
        p.bounds + (static_cast<int64_t>(ok ? id : 0) * p.Hkv + h) * (4 * D) + (threadIdx.x & 31) * (V * 2);
    uint32_t w[2][V / 2];
    load_words<V * 2>(b, w[0]);
    load_words<V * 2>(b + 2 * D, w[1]);
    Unpack<T, V>::run(w[0], lo);
    Unpack<T, V>::run(w[1], hi);
    return ok;
}

// The binary32 scores of four blocks by one warp; lane l gets that of block j[l / 8].
// A lane's four (block, channel) strips against the eight query heads are 32 sums,
// which one reduce-scatter (31 shuffles, not 5 a sum) leaves one a lane.  An
// element's sum takes at most D / 32 - 1 + 5 = 8 additions of exact products, each
// within 2^-24 of the sum of magnitudes.  q: the G query rows in shared memory.
template <int D, typename T>
__device__ __forceinline__ float four_scores(const SelectParams& p, const float* q, int s, int h, const int (&j)[4]) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    float lo[4][V], hi[4][V], v[32];
    bool ok = false;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        const bool in = lane_bounds<D, T>(p, s, h, j[n], lo[n], hi[n]);
        if ((lane >> 3) == n) ok = in;
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
#pragma unroll
        for (int n = 0; n < 4; ++n) v[8 * n + g] = 0.f;
        if (g < p.G) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float x = q[g * D + lane * V + i];
#pragma unroll
                for (int n = 0; n < 4; ++n) v[8 * n + g] = fmaf(x, x < 0.f ? lo[n][i] : hi[n][i], v[8 * n + g]);
            }
        }
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int k = 0; k < m; ++k) {
            const float send = upper ? v[k] : v[k + m], keep = upper ? v[k + m] : v[k];
            v[k] = keep + __shfl_xor_sync(kFull, send, m);
        }
    }
    float best = (lane & 7) < p.G ? v[0] : -INFINITY;
    if (!(best == best)) best = -INFINITY;  // NaN is dropped
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) best = fmaxf(best, __shfl_xor_sync(kFull, best, m));
    return ok ? best : -INFINITY;
}

// The score of block j in 64 bits, by one warp: products of 16-bit values are
// exact, and so, but for extreme ranges, are their sums.
template <int D, typename T>
__device__ __forceinline__ double exact_score(const SelectParams& p, const float* q, int s, int h, int j) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    float lo[V], hi[V];
    const bool ok = lane_bounds<D, T>(p, s, h, j, lo, hi);
    double best = -HUGE_VAL;
    for (int g = 0; g < p.G; ++g) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = q[g * D + lane * V + i];
            sum += static_cast<double>(x) * static_cast<double>(x < 0.f ? lo[i] : hi[i]);
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(kFull, sum, m);
        if (sum > best) best = sum;  // NaN is dropped
    }
    return ok ? best : -HUGE_VAL;
}

// One CTA per (KV head, sequence): the n blocks of the highest scores, in
// ascending order of their numbers, ties to the lowest number.
//
// The binary32 scores decide all but a border band.  Every product in them is
// exact; an MMA adds 16 of them to its accumulator, aligned to the largest
// addend, with an error of at most 17 * 2^-23 of it, and a score is D / 8 MMAs
// in two chains of at most 8, so with A = max_g |q_g|_1 * max |bound| it is within
// 8 * 17 * 2^-23 A + 2^-23 A < 2^-15 A of the true score.  eps = 2^-14 A covers it
// twice; 2^-117 more covers products and sums below 2^-126, each of which may be
// flushed (2 D of them, twice).  A histogram over the scores' range finds the bin that holds the k-th
// highest, zooming in while the bin is wide and full; with [tl, th] around the
// scores in it, a block above th + 2 eps is in and one below tl - 2 eps is out,
// and the few between them are scored again, in binary32 with a far smaller
// bound and, where that leaves an order open, in 64 bits, and ranked by (score,
// number).  So the answer is that of exact arithmetic whatever the order of the
// binary32 sums.  Where A is not below 2^126 they may have overflowed on the way
// to a finite score, and every block is scored in 64 bits.
//
// Bound by latency, a dozen barriers and three chains of loads: 5 us after the
// scores for 8 rows of 512 blocks, 13 us for 256 rows of 2000.  64-bit scores for
// the whole band (13 blocks on average) took 20 us more: the card's 64-bit rate is
// two FMAs a cycle and SM, and the binary32 pass leaves 0.16 of them a row.
template <int D, typename T>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    extern __shared__ __align__(16) float row_smem[];
    __shared__ int hist[kSelBins];
    __shared__ __align__(16) float qs[8 * D];
    __shared__ float redf[4][kSelWarps];
    __shared__ int redi[kSelWarps];
    __shared__ int near_id[kSelNear];
    __shared__ double near_y[kSelNear];
    __shared__ float near_f[kSelNear];
    __shared__ short tie[kSelNear];
    __shared__ int sh[5];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = static_cast<int64_t>(s) * p.Hkv + h;
    int32_t* out = p.selected + row * p.n;
    bool bad;
    const int nblk = row_blocks(p, s, bad);
    if (nblk <= p.n) {  // every block; not waiting for the scores is fine, none are read or written
        for (int i = tid; i < p.n; i += kSelThreads) out[i] = i < nblk ? i : -1;
        wait_primary_grid();
        return;
    }
    // the free range [f0, f1) and how many of it to keep: n >= sink + recent and nblk > n
    const int f0 = p.sink, f1 = nblk - p.recent, m = f1 - f0, k = p.n - p.sink - p.recent;
    // A: the largest |q_g|_1, while the scores are still being made
    float q1 = 0.f;
    for (int g = warp; g < p.G; g += kSelWarps) {
        const typename T::storage* q =
            reinterpret_cast<const typename T::storage*>(p.q) + (static_cast<int64_t>(s) * p.Hq + h * p.G + g) * D;
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const float x = to_float(q[lane + 32 * i]);
            qs[g * D + lane + 32 * i] = x;
            a += fabsf(x);
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) a += __shfl_xor_sync(kFull, a, x);
        q1 = fmaxf(q1, a);
    }
    for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
    if (tid == 0) sh[2] = sh[3] = sh[4] = 0;
    wait_primary_grid();
    float* sc = p.score + row * p.cols;
    const bool in_smem = nblk <= p.smem_cols;
    float a = INFINITY, b = -INFINITY, big = 0.f;
    for (int i = tid; i < (nblk + 15) / 16; i += kSelThreads) big = fmaxf(big, __ldcg(p.top + row * (p.cols / 16) + i));
    if (in_smem) {
        // columns past nblk up to the next tile's end are written too (-inf)
        const float4* src = reinterpret_cast<const float4*>(sc);
        float4* dst = reinterpret_cast<float4*>(row_smem);
        const int quads = (nblk + 3) / 4;
#pragma unroll 4
        for (int i = tid; i < quads; i += kSelThreads) {
            const float4 v = __ldcg(src + i);
            dst[i] = v;
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = 4 * i + e >= f0 && 4 * i + e < f1;
                if (in && x[e] > -INFINITY) a = fminf(a, x[e]);
                if (in) b = fmaxf(b, x[e]);
            }
        }
        sc = row_smem;
    } else {
        for (int i = f0 + tid; i < f1; i += kSelThreads) {
            const float x = sc[i];
            if (x > -INFINITY) a = fminf(a, x);
            b = fmaxf(b, x);
        }
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) {
        a = fminf(a, __shfl_xor_sync(kFull, a, x));
        b = fmaxf(b, __shfl_xor_sync(kFull, b, x));
        big = fmaxf(big, __shfl_xor_sync(kFull, big, x));
    }
    if (lane == 0) {
        redf[0][warp] = a;
        redf[1][warp] = b;
        redf[2][warp] = big;
        redf[3][warp] = q1;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        a = fminf(a, redf[0][w]);
        b = fmaxf(b, redf[1][w]);
        big = fmaxf(big, redf[2][w]);
        q1 = fmaxf(q1, redf[3][w]);
    }
    const float A = q1 * big;  // from 2^126 on sums may have overflowed: every block in the band
    const float eps2 = A < 0x1p126f ? 2.f * (0x1p-14f * A + 0x1p-117f) : INFINITY;

    float thr = INFINITY;  // blocks above it are in
    if (k > 0) {
        if (!(a <= b)) a = b;  // no finite score at all
        for (int round = 0; round < 4; ++round) {
            const float scale = kSelBins / (b - a);
            if (!(b > a) || !(scale < INFINITY) || !(scale > 0.f)) break;
            if (round) {
                for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
                if (tid == 0) sh[4] = 0;
                __syncthreads();
            }
            int over = 0;  // blocks known to score over b
#pragma unroll 4
            for (int i = f0 + tid; i < f1; i += kSelThreads) {
                const float x = sc[i];
                if (x > b)
                    ++over;
                else if (x >= a)
                    atomicAdd(&hist[min(kSelBins - 1, static_cast<int>((x - a) * scale))], 1);
            }
            if (round) {
                over = __reduce_add_sync(kFull, over);
                if (lane == 0 && over) atomicAdd(&sh[4], over);
            }
            __syncthreads();
            // the bin of the k-th highest: scan from the top, four bins a thread
            constexpr int PB = kSelBins / kSelThreads;
            const int top_bin = kSelBins - 1 - PB * tid;
            int c[PB], sum = 0;
#pragma unroll
            for (int i = 0; i < PB; ++i) sum += c[i] = hist[top_bin - i];
            int before = sh[4] + cta_scan(sum, redi);
            if (tid == 0) sh[0] = -1;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                if (before < k && before + c[i] >= k) {
                    sh[0] = top_bin - i;
                    sh[1] = c[i];
                }
                before += c[i];
            }
            __syncthreads();
            const int t = sh[0];
            if (t < 0) {  // the k-th is below every finite score
                b = a;
                break;
            }
            // the bin's edges, out by 2^-8 of a bin: (x - a) * scale is within 2^-12 of a bin
            const float lo = a + (t - 0x1p-8f) / scale, hi = a + (t + 1 + 0x1p-8f) / scale;
            a = fmaxf(a, lo);
            b = fminf(b, hi);
            if (sh[1] <= 16 || b - a <= eps2) break;
            __syncthreads();  // sh and hist are written again
        }
        float low = a - eps2;
        thr = b + eps2;
        if (!(low > -INFINITY) || !(thr < INFINITY)) {  // no usable bound: all in the band
            low = -INFINITY;
            thr = INFINITY;
        }
        // ---- sure of being in, and the band
        int sure = 0;
#pragma unroll 4
        for (int i = f0 + tid; i < f1; i += kSelThreads) {
            const float x = sc[i];
            if (x > thr) {
                ++sure;
            } else if (x >= low) {
                const int at = atomicAdd(&sh[3], 1);
                if (at < kSelNear) near_id[at] = i;
            }
        }
        sure = __reduce_add_sync(kFull, sure);
        if (lane == 0 && sure) atomicAdd(&sh[2], sure);
        __syncthreads();
        sure = sh[2];
        int band = sh[3];
        const int want = k - sure;
        bool listed = band <= kSelNear;
        if (band < want) {  // blocks without a usable score fill up
            low = -INFINITY;
            band = m - sure;
            listed = false;
        }
        __syncthreads();  // sh is written again
        if (band == want) {  // all of the band
            for (int i = f0 + tid; i < f1; i += kSelThreads) {
                const float x = sc[i];
                if (x <= thr && x >= low) sc[i] = INFINITY;
            }
        } else if (listed) {
            // binary32 first, each within 8 * 2^-24 A: twice that and its double is eps2 / 64
            for (int i = 4 * warp; i < band; i += 4 * kSelWarps) {
                int j[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) j[u] = i + u < band ? near_id[i + u] : -1;
                const float y = four_scores<D, T>(p, qs, s, h, j);
                if ((lane & 7) == 0 && i + (lane >> 3) < band) near_f[i + (lane >> 3)] = y;
            }
            if (tid == 0) sh[3] = sh[2] = 0;
            __syncthreads();
            const float e2 = eps2 * 0x1p-6f;
            for (int i = tid; i < band; i += kSelThreads) {
                const float y = near_f[i];
                int over = 0, near_or_over = 0;
                for (int j = 0; j < band; ++j) {
                    over += near_f[j] > y + e2;
                    near_or_over += !(near_f[j] < y - e2);
                }
                const bool in = near_or_over <= want && e2 < INFINITY, off = over >= want && e2 < INFINITY;
                if (in) atomicAdd(&sh[2], 1);
                if (in || off)
                    sc[near_id[i]] = in ? INFINITY : -INFINITY;
                else
                    tie[atomicAdd(&sh[3], 1)] = i;
            }
            __syncthreads();
            const int ties = sh[3], left = want - sh[2];
            if (ties > 0) {  // the few that binary32 cannot order: 64 bits
                for (int i = warp; i < ties; i += kSelWarps) {
                    const double y = exact_score<D, T>(p, qs, s, h, near_id[tie[i]]);
                    if (lane == 0) near_y[i] = y;
                }
                __syncthreads();
                for (int i = tid; i < ties; i += kSelThreads) {
                    const double y = near_y[i];
                    const int at = near_id[tie[i]];
                    int rank = 0;
                    for (int j = 0; j < ties; ++j) rank += near_y[j] > y || (near_y[j] == y && near_id[tie[j]] < at);
                    sc[at] = rank < left ? INFINITY : -INFINITY;
                }
            }
        } else {
            // many near the border (equal scores): radix selection of the want-th
            // highest 64-bit score, then the lowest numbers among those equal to it
            double* ex = p.exact + row * p.cols;
            for (int i = f0 + warp; i < f1; i += kSelWarps) {
                const float x = sc[i];
                if (!(x <= thr && x >= low)) continue;
                const double y = exact_score<D, T>(p, qs, s, h, i);
                if (lane == 0) ex[i] = y;
            }
            __syncthreads();
            uint64_t prefix = 0, mask = 0;
            int left = want;
            for (int shift = 56; shift >= 0; shift -= 8) {
                hist[tid] = 0;
                __syncthreads();
                for (int i = f0 + tid; i < f1; i += kSelThreads) {
                    const float x = sc[i];
                    if (!(x <= thr && x >= low)) continue;
                    const uint64_t o = order64(ex[i]);
                    if ((o & mask) == prefix) atomicAdd(&hist[(o >> shift) & 255], 1);
                }
                __syncthreads();
                const int c = hist[255 - tid];
                const int before = cta_scan(c, redi);
                if (before < left && before + c >= left) {
                    sh[0] = 255 - tid;
                    sh[1] = left - before;
                }
                __syncthreads();
                prefix |= static_cast<uint64_t>(sh[0]) << shift;
                mask |= 255ull << shift;
                left = sh[1];
                __syncthreads();
            }
            // `left` of the blocks whose score has these bits, lowest numbers first
            const int per = (m + kSelThreads - 1) / kSelThreads;
            const int i0 = f0 + tid * per, i1 = min(f1, i0 + per);
            int same = 0;
            for (int i = i0; i < i1; ++i) same += sc[i] <= thr && sc[i] >= low && order64(ex[i]) == prefix;
            int at = cta_scan(same, redi);
            for (int i = i0; i < i1; ++i) {
                const float x = sc[i];
                if (!(x <= thr && x >= low)) continue;
                const uint64_t o = order64(ex[i]);
                const bool in = o > prefix || (o == prefix && at++ < left);
                sc[i] = in ? INFINITY : -INFINITY;
            }
        }
        __syncthreads();
    }
    // ---- the kept blocks in ascending order: a warp takes a run of 32-block groups
    const auto kept = [&](int i) {
        return i < nblk && (i < f0 || i >= f1 || (k > 0 && (sc[i] > thr || sc[i] == INFINITY)));
    };
    const int groups = ((nblk + 31) / 32 + kSelWarps - 1) / kSelWarps;
    const int g0 = warp * groups;
    int mine = 0;
#pragma unroll 4
    for (int g = g0; g < g0 + groups && g * 32 < nblk; ++g) mine += __popc(__ballot_sync(kFull, kept(g * 32 + lane)));
    if (lane == 0) redi[warp] = mine;
    __syncthreads();
    int at = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w)
        if (w < warp) at += redi[w];
#pragma unroll 4
    for (int g = g0; g < g0 + groups && g * 32 < nblk; ++g) {
        const bool keep = kept(g * 32 + lane);
        const uint32_t votes = __ballot_sync(kFull, keep);
        const int to = at + __popc(votes & ((1u << lane) - 1u));
        if (keep && to < p.n) out[to] = g * 32 + lane;
        at += __popc(votes);
    }
}

template <int D, typename T>
cudaError_t launch_select(const SelectParams& p, cudaStream_t st) {
    const int64_t units = static_cast<int64_t>((p.cols / 16 + p.tiles - 1) / p.tiles) * p.Hkv;
    constexpr int kScoreSmem = ScoreCfg<D>::kBytes;
    static bool configured[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(block_score_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(select_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemCols * 4);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    e = launch_maybe_pdl(true, block_score_kernel<D, T>, dim3(static_cast<unsigned>((units + 3) / 4), p.S), dim3(128),
                         kScoreSmem, st, p);
    if (e != cudaSuccess) return e;
    const size_t smem = static_cast<size_t>(p.smem_cols) * 4;
    return launch_maybe_pdl(true, select_kernel<D, T>, dim3(p.Hkv, p.S), dim3(kSelThreads), smem, st, p);
}

template <int D, typename OT>
cudaError_t launch_bounds_of(int kv, dim3 grid, cudaStream_t st, const unsigned char* kc, const int32_t* tables, int MB,
                             const int32_t* lens, const int32_t* fresh, int max_new, const pkv_cache_desc* d,
                             unsigned char* bounds, unsigned int* err) {
    void (*kern)(const unsigned char*, const int32_t*, int, const int32_t*, const int32_t*, int, int, int, float,
                 unsigned char*, unsigned int*) = nullptr;
    switch (kv) {
    case PKV_F16: kern = key_bounds_kernel<D, PKV_F16, F16>; break;
    case PKV_BF16: kern = key_bounds_kernel<D, PKV_BF16, BF16>; break;
    case PKV_FP8_E4M3: kern = key_bounds_kernel<D, PKV_FP8_E4M3, OT>; break;
    case PKV_INT8: kern = key_bounds_kernel<D, PKV_INT8, OT>; break;
    default: kern = key_bounds_kernel<D, PKV_INT4, OT>; break;
    }
    return launch_maybe_pdl(true, kern, grid, dim3(128), 0, st, kc, tables, MB, lens, fresh, max_new, d->num_blocks,
                            d->num_kv_heads, d->k_scale, bounds, err);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Checks that the three calls share.
pkv_status check_desc(const pkv_cache_desc* d, int32_t num_seqs, int32_t max_blocks_per_seq) {
    if (!d || num_seqs < 0 || max_blocks_per_seq <= 0) return PKV_ERR_INVALID;
    if (d->num_blocks <= 0 || d->num_kv_heads <= 0 || d->head_size <= 0 || d->block_size <= 0) return PKV_ERR_INVALID;
    if (!known_kv_dtype(d->kv_dtype)) return PKV_ERR_INVALID;
    if (d->kv_dtype == PKV_FP8_E4M3 && !(d->k_scale > 0.f && d->v_scale > 0.f)) return PKV_ERR_INVALID;
    if (d->block_size != kBlockSize || (d->head_size != 64 && d->head_size != 128)) return PKV_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || d->num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
    if (max_blocks_per_seq > 0x7fffffff / kBlockSize) return PKV_ERR_UNSUPPORTED;  // positions are 32-bit
    return PKV_OK;
}

bool group_ok(int32_t num_q_heads, const pkv_cache_desc* d, pkv_status* st) {
    *st = PKV_ERR_INVALID;
    if (num_q_heads <= 0 || num_q_heads % d->num_kv_heads) return false;
    const int G = num_q_heads / d->num_kv_heads;
    *st = PKV_ERR_UNSUPPORTED;
    return G == 1 || G == 2 || G == 4 || G == 8;
}

struct SelectLayout {
    int64_t cols, top_off, exact_off, bytes;
};
SelectLayout select_layout(int64_t S, int64_t Hkv, int64_t max_seq_len) {
    const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    SelectLayout l{};
    l.cols = cdiv(max_seq_len > 0 ? cdiv(max_seq_len, kBlockSize) : 1, 16) * 16;
    const int64_t rows = S * Hkv;
    l.top_off = up(rows * l.cols * 4);
    l.exact_off = l.top_off + up(rows * (l.cols / 16) * 4);
    l.bytes = l.exact_off + up(rows * l.cols * 8);
    return l;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_paged_key_bounds(const void* k_cache, const pkv_cache_desc* d, const int32_t* block_tables,
                                           int32_t max_blocks_per_seq, const int32_t* seq_lens, const int32_t* new_lens,
                                           int32_t max_new_len, int32_t num_seqs, void* bounds, int32_t bounds_dtype,
                                           void* stream) {
    const pkv_status c = check_desc(d, num_seqs, max_blocks_per_seq);
    if (c != PKV_OK) return c;
    if (max_new_len < 0 || (bounds_dtype != PKV_F16 && bounds_dtype != PKV_BF16)) return PKV_ERR_INVALID;
    if ((d->kv_dtype == PKV_F16 || d->kv_dtype == PKV_BF16) && bounds_dtype != d->kv_dtype) return PKV_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_new_len) > static_cast<int64_t>(max_blocks_per_seq) * kBlockSize) return PKV_ERR_INVALID;
    if (num_seqs == 0 || max_new_len == 0) return PKV_OK;
    if (!k_cache || !block_tables || !seq_lens || !bounds) return PKV_ERR_INVALID;
    if (!aligned(k_cache, 16) || !aligned(bounds, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(new_lens, 4))
        return PKV_ERR_INVALID;
    unsigned int* err = error_word();
    if (!err) return PKV_ERR_CUDA;
    // n new tokens reach into at most (n + 14) / 16 + 1 blocks
    const int64_t reach = (static_cast<int64_t>(max_new_len) + 14) / kBlockSize + 1;
    const dim3 grid(static_cast<unsigned>(reach < max_blocks_per_seq ? reach : max_blocks_per_seq),
                    static_cast<unsigned>(num_seqs));
    const auto* kc = static_cast<const unsigned char*>(k_cache);
    auto* out = static_cast<unsigned char*>(bounds);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf = bounds_dtype == PKV_BF16;
    cudaError_t e;
    if (d->head_size == 128)
        e = bf ? launch_bounds_of<128, BF16>(d->kv_dtype, grid, st, kc, block_tables, max_blocks_per_seq, seq_lens, new_lens,
                                             max_new_len, d, out, err)
               : launch_bounds_of<128, F16>(d->kv_dtype, grid, st, kc, block_tables, max_blocks_per_seq, seq_lens, new_lens,
                                            max_new_len, d, out, err);
    else
        e = bf ? launch_bounds_of<64, BF16>(d->kv_dtype, grid, st, kc, block_tables, max_blocks_per_seq, seq_lens, new_lens,
                                            max_new_len, d, out, err)
               : launch_bounds_of<64, F16>(d->kv_dtype, grid, st, kc, block_tables, max_blocks_per_seq, seq_lens, new_lens,
                                           max_new_len, d, out, err);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" size_t pkv_select_blocks_workspace_bytes(int32_t num_seqs, int32_t num_kv_heads, int32_t max_seq_len) {
    if (num_seqs < 0 || num_kv_heads <= 0 || max_seq_len < 0) return 0;
    return static_cast<size_t>(select_layout(num_seqs, num_kv_heads, max_seq_len).bytes);
}

extern "C" pkv_status pkv_select_blocks(const void* q, int32_t q_dtype, int32_t num_seqs, int32_t num_q_heads,
                                        const void* bounds, const pkv_cache_desc* d, const int32_t* block_tables,
                                        int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t max_seq_len,
                                        int32_t num_selected, int32_t sink_blocks, int32_t recent_blocks,
                                        int32_t* selected, void* workspace, size_t workspace_bytes, void* stream) {
    const pkv_status c = check_desc(d, num_seqs, max_blocks_per_seq);
    if (c != PKV_OK) return c;
    if ((q_dtype != PKV_F16 && q_dtype != PKV_BF16) || max_seq_len < 0) return PKV_ERR_INVALID;
    if (num_selected <= 0 || sink_blocks < 0 || recent_blocks < 0 ||
        static_cast<int64_t>(sink_blocks) + recent_blocks > num_selected)
        return PKV_ERR_INVALID;
    if (static_cast<int64_t>(max_seq_len) > static_cast<int64_t>(max_blocks_per_seq) * kBlockSize) return PKV_ERR_INVALID;
    pkv_status g;
    if (!group_ok(num_q_heads, d, &g)) return g;
    if ((d->kv_dtype == PKV_F16 || d->kv_dtype == PKV_BF16) && q_dtype != d->kv_dtype) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !bounds || !block_tables || !seq_lens || !selected) return PKV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(block_tables, 4) || !aligned(seq_lens, 4) ||
        !aligned(selected, 4))
        return PKV_ERR_INVALID;
    const SelectLayout l = select_layout(num_seqs, d->num_kv_heads, max_seq_len);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < static_cast<size_t>(l.bytes)) return PKV_ERR_WORKSPACE;
    SelectParams p{};
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    p.q = q;
    p.bounds = static_cast<const unsigned char*>(bounds);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.selected = selected;
    p.score = reinterpret_cast<float*>(ws);
    p.top = reinterpret_cast<float*>(ws + l.top_off);
    p.exact = reinterpret_cast<double*>(ws + l.exact_off);
    p.S = num_seqs;
    p.Hq = num_q_heads;
    p.Hkv = d->num_kv_heads;
    p.G = num_q_heads / d->num_kv_heads;
    p.MB = max_blocks_per_seq;
    p.NB = d->num_blocks;
    p.cols = static_cast<int>(l.cols);
    p.n = num_selected;
    p.sink = sink_blocks;
    p.recent = recent_blocks;
    // tiles a warp takes in a run: the number whose whole rounds of resident CTAs
    // cost least, a run's start counted as three tiles
    const int64_t row_tiles = l.cols / 16;
    const int64_t slots = (d->head_size == 128 ? ScoreCfg<128>::kCtasPerSm : ScoreCfg<64>::kCtasPerSm) *
                          static_cast<int64_t>(num_sms());
    int64_t best = INT64_MAX;
    for (int run = 1; run <= 64; ++run) {
        const int64_t ctas = cdiv(cdiv(row_tiles, run) * p.Hkv, 4) * p.S, cost = cdiv(ctas, slots) * (run + 3);
        if (cost < best) {
            best = cost;
            p.tiles = run;
        }
    }
    p.smem_cols = static_cast<int>(std::min<int64_t>(l.cols, kSmemCols));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf = q_dtype == PKV_BF16;
    cudaError_t e;
    if (d->head_size == 128)
        e = bf ? launch_select<128, BF16>(p, st) : launch_select<128, F16>(p, st);
    else
        e = bf ? launch_select<64, BF16>(p, st) : launch_select<64, F16>(p, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// List entries per partition of the automatic choice: the dense decode's rule for
// a sequence of the list's length, whose least is 16 blocks, but 8 where 8 still
// leave the launch within one CTA an SM: then a CTA's chain of loads is what the
// call waits for, and halving it gains more than the merge's doubled rows cost.
// 1 sequence x 8 KV heads x 128 blocks, bf16: 5.8 us against 7.2 (128 and 64
// CTAs), int8 5.5 against 6.3; 1 x 1 x 400, bf16: 5.9 against 7.0; with more CTAs, 2
// x 8 x 128, int8: 6.6 against 6.3 (bf16 6.8 against 7.2).  Four blocks: 6.2, 6.1,
// 6.1.  A workspace that holds partitions of 16 blocks only is taken too, with those.
constexpr int kSmallPartition = 8, kSmallLaunch = 152;

static bool small_lists(int64_t S, int64_t Hkv, int n) {
    return n > kAutoMinPartition / kBlockSize && S * Hkv <= kSmallLaunch &&
           S * Hkv * cdiv(n, kSmallPartition) <= kSmallLaunch;
}

static int auto_list_partition(int S, int Hq, const pkv_cache_desc* d, int n, size_t workspace_bytes) {
    if (small_lists(S, d->num_kv_heads, n) &&
        workspace_bytes >= partials_bytes(S, Hq, d->head_size, cdiv(n, kSmallPartition)))
        return kSmallPartition;
    const int tokens = n * kBlockSize;
    return (is_int_pool(d->kv_dtype) ? auto_partition_int(S, d->num_kv_heads, tokens, d->kv_dtype, d->head_size)
                                     : auto_partition(S, d->num_kv_heads, tokens, false)) /
           kBlockSize;
}

extern "C" size_t pkv_decode_sparse_workspace_bytes(int32_t num_seqs, int32_t num_q_heads, int32_t head_size,
                                                    int32_t num_selected, int32_t partition_blocks) {
    if (num_seqs < 0 || num_q_heads <= 0 || head_size <= 0 || num_selected <= 0 || partition_blocks < 0) return 0;
    // one KV head gives the automatic choice its smallest partitions
    const int per = partition_blocks > 0 ? partition_blocks : small_lists(num_seqs, 1, num_selected) ? kSmallPartition
                                                            : kAutoMinPartition / kBlockSize;
    const int64_t NP = cdiv(num_selected, per);
    return NP <= 1 ? 0 : partials_bytes(num_seqs, num_q_heads, head_size, NP);
}

extern "C" pkv_status pkv_paged_attention_decode_sparse(const void* q, int32_t q_dtype, int32_t num_seqs,
                                                        int32_t num_q_heads, const void* k_cache, const void* v_cache,
                                                        const pkv_cache_desc* d, const int32_t* block_tables,
                                                        int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                                        const int32_t* selected, int32_t num_selected, float scale,
                                                        void* out, void* workspace, size_t workspace_bytes,
                                                        int32_t partition_blocks, void* stream) {
    const pkv_status c = check_desc(d, num_seqs, max_blocks_per_seq);
    if (c != PKV_OK) return c;
    if ((q_dtype != PKV_F16 && q_dtype != PKV_BF16) || !(scale == scale)) return PKV_ERR_INVALID;
    if (num_selected <= 0 || partition_blocks < 0 || partition_blocks > 0x7fffffff / kBlockSize ||
        num_selected > 0x7fffffff / kBlockSize)
        return PKV_ERR_INVALID;
    pkv_status g;
    if (!group_ok(num_q_heads, d, &g)) return g;
    if ((d->kv_dtype == PKV_F16 || d->kv_dtype == PKV_BF16) && q_dtype != d->kv_dtype) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!q || !k_cache || !v_cache || !block_tables || !seq_lens || !selected || !out) return PKV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(seq_lens, 4) || !aligned(selected, 4))
        return PKV_ERR_INVALID;
    const int G = num_q_heads / d->num_kv_heads;
    const int per = partition_blocks > 0
                        ? partition_blocks
                        : auto_list_partition(num_seqs, num_q_heads, d, num_selected, workspace_bytes);
    const int64_t NP = cdiv(num_selected, per);
    const size_t need = NP > 1 ? partials_bytes(num_seqs, num_q_heads, d->head_size, NP) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return PKV_ERR_WORKSPACE;
    DecodeParams p{};
    p.err = error_word();
    if (!p.err) return PKV_ERR_CUDA;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.out = out;
    p.S = num_seqs;
    p.Hq = num_q_heads;
    p.Hkv = d->num_kv_heads;
    p.D = d->head_size;
    p.NB = d->num_blocks;
    p.MB = max_blocks_per_seq;
    p.P = per * kBlockSize;
    p.NP = static_cast<int32_t>(NP);
    const bool fp8 = d->kv_dtype == PKV_FP8_E4M3;
    p.qk_scale = scale * 1.4426950408889634f * (fp8 ? d->k_scale : 1.f);
    p.v_scale = fp8 ? d->v_scale : 1.f;
    p.selected = selected;
    p.nsel = num_selected;
    if (need > 0) partials_layout(p, workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (is_int_pool(d->kv_dtype)) {
        e = d->kv_dtype == PKV_INT8 ? launch_decode_int8(p, G, q_dtype, st) : launch_decode_int4(p, G, q_dtype, st);
    } else {
        // the kernel that the dense decode of this shape would use
        const int64_t pool_rows = static_cast<int64_t>(d->num_blocks) * d->num_kv_heads * kBlockSize;
        CUtensorMap tk, tv;
        const bool mma = d->head_size == 128 && G >= 2 && pool_rows <= 0x7fffffff;
        if (mma && (!encode_pool_map(&tk, k_cache, fp8 ? 1 : 2, pool_rows, d->head_size) ||
                    !encode_pool_map(&tv, v_cache, fp8 ? 1 : 2, pool_rows, d->head_size)))
            return PKV_ERR_CUDA;
        const CUtensorMap* mk = mma ? &tk : nullptr;
        const CUtensorMap* mv = mma ? &tv : nullptr;
        if (fp8)
            e = launch_decode_sparse_fp8(p, G, q_dtype, mk, mv, st);
        else
            e = d->kv_dtype == PKV_F16 ? launch_decode_sparse_f16(p, G, mk, mv, st)
                                       : launch_decode_sparse_bf16(p, G, mk, mv, st);
    }
    if (e != cudaSuccess) return PKV_ERR_CUDA;
    if (NP > 1 && launch_merge(p, q_dtype, st) != cudaSuccess) return PKV_ERR_CUDA;
    return PKV_OK;
}
