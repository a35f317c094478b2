// evict.cu -- a cache cut to a budget of keys by accumulated attention weight.
//
// A sequence of L keys is cut to n = min(L, budget): every KV head keeps its
// first `sink` and last `recent` positions and, of the others, those with the
// most accumulated weight (pkv_attn_decode_weights), and its kept rows move to
// positions 0 .. n - 1 in their old order.  Softmax attention does not depend
// on the order of the keys, and each head reads only its own rows, so heads
// may keep different positions while the sequence keeps one block table and
// one length.
//
//  * evict_select_kernel: the n-th largest weight of a row by radix selection
//    on the order-preserving integer image of the floats (11 + 11 + 10 bits),
//    then one ordered pass that writes the kept positions.
//  * evict_compact_kernel, evict_compact_i8_kernel: the moves, in place.  Row
//    i comes from position kept[i] >= i and kept ascends, so a chunk of rows
//    whose sources were all read can be written without touching a source of
//    any later chunk; chunks of one (sequence, head) are taken in order, each
//    one's loads before its stores.
#include "launch.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

struct SelectParams {
    const float *w;
    int64_t seq_stride, head_stride;
    const int32_t *seq_lens;
    int32_t hkv;
    int64_t max_keys;
    int32_t budget, sink, recent;
    int32_t *kept;
    int32_t *new_lens;
    int32_t *err;
};

// Integers that order as the floats do (-0 as +0), NaN above +inf.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.f);
    if (f != f) return 0xFFFFFFFEu;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive block-wide prefix of two ints per thread; totals in *ta, *tb.
__device__ __forceinline__ void block_prefix2(int &a, int &b, int *ta, int *tb, int (*s)[kSelWarps]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) {
        s[0][warp] = x;
        s[1][warp] = y;
    }
    __syncthreads();
    if (warp == 0) {
        int p = s[0][lane], q = s[1][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, p, o), v = __shfl_up_sync(0xffffffffu, q, o);
            if (lane >= o) {
                p += u;
                q += v;
            }
        }
        s[0][lane] = p;
        s[1][lane] = q;
    }
    __syncthreads();
    a = x - a + (warp ? s[0][warp - 1] : 0);
    b = y - b + (warp ? s[1][warp - 1] : 0);
    *ta = s[0][kSelWarps - 1];
    *tb = s[1][kSelWarps - 1];
    __syncthreads();
}

// One CTA per (sequence, KV head).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
    __shared__ int s_hist[kBins];
    __shared__ int s_scan[2][kSelWarps];
    __shared__ int s_bin, s_need;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int64_t seq = row / p.hkv;
    const int h = (int)(row - seq * p.hkv);
    const int L = p.seq_lens[seq];
    int32_t *kept = p.kept + row * p.budget;
    const bool bad = L < 0 || L > p.max_keys;
    if (tid == 0 && h == 0) {
        if (bad) set_err(p.err, PKV_DEVERR_LENGTH);
        p.new_lens[seq] = bad || L < p.budget ? L : p.budget;
    }
    if (bad || L <= p.budget) {  // nothing goes
        for (int i = tid; i < p.budget; i += kSelThreads) kept[i] = !bad && i < L ? i : -1;
        return;
    }
    const float *w = p.w + seq * p.seq_stride + h * p.head_stride;
    const int tail = L - p.recent;
    auto key = [&](int t) -> uint32_t { return t < p.sink || t >= tail ? 0xFFFFFFFFu : order_key(w[t]); };

    // the budget-th largest key, digit by digit
    uint32_t prefix = 0, mask = 0;
    int need = p.budget;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        for (int t = tid; t < L; t += kSelThreads) {
            const uint32_t k = key(t);
            if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & digits], 1);
        }
        __syncthreads();
        // thread i holds bins 2047 - 2i and 2046 - 2i: an exclusive prefix counts the keys above
        const int hi = kBins - 1 - 2 * tid;
        const int c0 = s_hist[hi], c1 = s_hist[hi - 1];
        int above = c0 + c1, dummy = 0, t0, t1;
        block_prefix2(above, dummy, &t0, &t1, s_scan);
        if (above < need && need <= above + c0 + c1) {
            const bool first = need <= above + c0;
            s_bin = first ? hi : hi - 1;
            s_need = need - above - (first ? 0 : c0);
        }
        __syncthreads();
        prefix |= (uint32_t)s_bin << shift;
        mask |= digits << shift;
        need = s_need;
        __syncthreads();
    }
    // keys above `prefix` stay, and the first `need` of those equal to it; a
    // warp takes a contiguous run of positions
    const int seg = ((L + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int a = min(L, warp * seg), b = min(L, a + seg);
    int gt = 0, eq = 0;
    for (int t = a + lane; t < b; t += 32) {
        const uint32_t k = key(t);
        gt += k > prefix;
        eq += k == prefix;
    }
    int ta, tb;
    block_prefix2(gt, eq, &ta, &tb, s_scan);
    gt = __shfl_sync(0xffffffffu, gt, 0);
    eq = __shfl_sync(0xffffffffu, eq, 0);
    int at = gt + min(eq, need);
    for (int t0 = a; t0 < b; t0 += 32) {
        const int t = t0 + lane;
        const uint32_t k = t < b ? key(t) : 0u;
        const unsigned me = 1u << lane, below = me - 1;
        const unsigned same = __ballot_sync(0xffffffffu, t < b && k == prefix);
        const bool take = t < b && (k > prefix || (k == prefix && eq + __popc(same & below) < need));
        const unsigned taken = __ballot_sync(0xffffffffu, take);
        if (take) kept[at + __popc(taken & below)] = t;
        at += __popc(taken);
        eq += __popc(same);
    }
}

// ---- moves ---------------------------------------------------------------------

constexpr int kMoveThreads = 512;
constexpr int kMoveRows = 16;                               // rows per warp and chunk
constexpr int kChunk = kMoveRows * kMoveThreads / 32;      // rows per chunk

struct CompactParams {
    void *k, *v;                 // pools
    float *k_scale, *v_scale;    // int8 caches
    const int32_t *tables;
    int32_t max_blocks;
    const int32_t *seq_lens;
    const int32_t *kept;
    int32_t budget;
    int32_t num_blocks, block_size, hkv;
    float *w;                    // accumulated weights, or NULL
    int64_t seq_stride, head_stride;
    int32_t chunk;               // rows per chunk (int8: whole blocks)
    int32_t *err;
};

// Where row i of (sequence, head) comes from and goes to: token rows of the
// pool, or src < 0 for a row that is not moved because its data is bad.
struct Move {
    int64_t src, dst;
    int32_t from;
};

__device__ __forceinline__ int64_t pool_row(const CompactParams &p, const int32_t *trow, int t) {
    const int lb = t / p.block_size;
    const int phys = trow[lb];
    if (phys < 0 || phys >= p.num_blocks) return -1;
    return (int64_t)phys * p.block_size + (t - lb * p.block_size);
}

__device__ __forceinline__ Move find_move(const CompactParams &p, const int32_t *kept, const int32_t *trow, int i, int L) {
    Move m;
    m.from = kept[i];
    m.src = m.dst = -1;
    if (m.from < i || m.from >= L || (i > 0 && kept[i - 1] >= m.from)) {
        set_err(p.err, PKV_DEVERR_KEEP);
        m.from = -1;
        return m;
    }
    m.src = pool_row(p, trow, m.from);
    m.dst = pool_row(p, trow, i);
    if (m.src < 0 || m.dst < 0) {
        set_err(p.err, PKV_DEVERR_BLOCK);
        m.src = m.dst = -1;
    }
    return m;
}

__device__ __forceinline__ int64_t shfl64(int64_t x, int lane) {
    return (int64_t)__shfl_sync(0xffffffffu, (long long)x, lane);
}

// One CTA per (sequence, KV head, K or V).  RB: bytes of a head's row.
template <int RB>
__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const CompactParams p) {
    constexpr int LPR = RB / 16;              // lanes per row
    constexpr int LOADS = kMoveRows * LPR / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = blockIdx.x;
    const int which = (int)(unit & 1);
    const int64_t head = unit >> 1;           // (sequence, KV head)
    const int64_t seq = head / p.hkv;
    const int h = (int)(head - seq * p.hkv);
    const int L = p.seq_lens[seq];
    if (L < 0 || (int64_t)L > (int64_t)p.max_blocks * p.block_size) {
        if (threadIdx.x == 0 && h == 0 && which == 0) set_err(p.err, PKV_DEVERR_LENGTH);
        return;
    }
    if (L <= p.budget) return;                // every key stays where it is
    const int n = p.budget;
    const int32_t *kept = p.kept + head * p.budget;
    const int32_t *trow = p.tables + seq * p.max_blocks;
    uint8_t *pool = static_cast<uint8_t *>(which ? p.v : p.k) + (int64_t)h * RB;
    const int64_t pitch = (int64_t)p.hkv * RB;
    float *w = p.w && which == 0 ? p.w + seq * p.seq_stride + h * p.head_stride : nullptr;
    for (int c0 = 0; c0 < n; c0 += kChunk) {
        const int i = c0 + warp * kMoveRows + lane;   // the row this lane looks up (lanes 0 .. 15)
        Move m;
        m.src = m.dst = -1;
        m.from = -1;
        if (lane < kMoveRows && i < n) m = find_move(p, kept, trow, i, L);
        if (m.from == i) m.src = -1;
        float wv = 0.f;
        if (w && m.from > i) wv = w[m.from];
        uint4 r[LOADS];
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int64_t src = shfl64(m.src, u * (32 / LPR) + lane / LPR);
            if (src >= 0) r[u] = *(reinterpret_cast<const uint4 *>(pool + src * pitch) + lane % LPR);
        }
        __syncthreads();  // every source of the chunk is read
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int from = u * (32 / LPR) + lane / LPR;
            const int64_t src = shfl64(m.src, from), dst = shfl64(m.dst, from);
            if (src >= 0) *(reinterpret_cast<uint4 *>(pool + dst * pitch) + lane % LPR) = r[u];
        }
        if (w && m.from > i) w[i] = wv;
    }
    if (w)
        for (int t = n + threadIdx.x; t < L; t += kMoveThreads) w[t] = 0.f;
}

__device__ __forceinline__ int32_t requantise(float x, float scale) {
    const float r = rintf(__fdiv_rn(x, scale));
    return (int32_t)fminf(fmaxf(r, -127.f), 127.f) & 255;
}

// The int8 cache: a block in which some row of the head moves gets a new
// scale, max|x| / 127 over its kept rows, and new codes, every decision in
// binary32 as in the quantised write (int8_write.cu).  Offsets kept[i] - i
// never fall, so a block is untouched exactly when its last kept row stays.
// A chunk is whole blocks; a warp's 16 rows lie in one block.
__global__ void __launch_bounds__(kMoveThreads) evict_compact_i8_kernel(const CompactParams p) {
    constexpr int RB = 128, LPR = 8, LOADS = kMoveRows * LPR / 32;
    __shared__ uint32_t s_max[3][kChunk / kMoveRows];  // three rounds: cleared a round ahead of its use
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = blockIdx.x;
    const int which = (int)(unit & 1);
    const int64_t head = unit >> 1;
    const int64_t seq = head / p.hkv;
    const int h = (int)(head - seq * p.hkv);
    const int L = p.seq_lens[seq];
    if (L < 0 || (int64_t)L > (int64_t)p.max_blocks * p.block_size) {
        if (threadIdx.x == 0 && h == 0 && which == 0) set_err(p.err, PKV_DEVERR_LENGTH);
        return;
    }
    if (L <= p.budget) return;
    const int n = p.budget;
    const int32_t *kept = p.kept + head * p.budget;
    const int32_t *trow = p.tables + seq * p.max_blocks;
    uint8_t *pool = static_cast<uint8_t *>(which ? p.v : p.k) + (int64_t)h * RB;
    float *scales = which ? p.v_scale : p.k_scale;
    const int64_t pitch = (int64_t)p.hkv * RB;
    float *w = p.w && which == 0 ? p.w + seq * p.seq_stride + h * p.head_stride : nullptr;
    if (threadIdx.x < 3 * (kChunk / kMoveRows)) s_max[0][threadIdx.x] = 0u;
    __syncthreads();
    int round = 0;
    for (int c0 = 0; c0 < n; c0 += p.chunk, round = round == 2 ? 0 : round + 1) {
        const int next = round == 2 ? 0 : round + 1;
        if (threadIdx.x < kChunk / kMoveRows) s_max[next][threadIdx.x] = 0u;
        const int local = warp * kMoveRows;             // first row of the warp in the chunk
        const int slot = local / p.block_size;          // its block in the chunk
        const int block_end = min(n, c0 + (slot + 1) * p.block_size);
        const int i = c0 + local + lane;
        const bool mine = local < p.chunk && c0 + local < n;
        const bool moved = mine && kept[block_end - 1] != block_end - 1;
        Move m;
        m.src = m.dst = -1;
        m.from = -1;
        float sc = 0.f, wv = 0.f;
        if (moved && lane < kMoveRows && i < n) {
            m = find_move(p, kept, trow, i, L);
            if (m.src >= 0) sc = scales[m.src / p.block_size * p.hkv + h];
            if (w && m.from > i) wv = w[m.from];
        }
        uint4 r[LOADS];
        float rs[LOADS];
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < LOADS; ++u) {
            const int from = u * (32 / LPR) + lane / LPR;
            const int64_t src = shfl64(m.src, from);
            rs[u] = __shfl_sync(0xffffffffu, sc, from);
            r[u] = make_uint4(0u, 0u, 0u, 0u);
            if (src >= 0) r[u] = *(reinterpret_cast<const uint4 *>(pool + src * pitch) + lane % LPR);
            const uint32_t words[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
            int big = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int b = 0; b < 4; ++b) big = max(big, abs((int)(int8_t)(words[j] >> (8 * b))));
            // |code| * |scale| rounds monotonically in |code|: the row's largest value
            top = fmaxf(top, __fmul_rn((float)big, fabsf(rs[u])));
        }
        if (moved) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (lane == 0) atomicMax(&s_max[round][slot], __float_as_uint(top));
        }
        __syncthreads();  // every source of the chunk is read, every block's maximum known
        if (moved) {
            const float scale = __fdiv_rn(__uint_as_float(s_max[round][slot]), 127.f);
#pragma unroll
            for (int u = 0; u < LOADS; ++u) {
                const int from = u * (32 / LPR) + lane / LPR;
                const int64_t dst = shfl64(m.dst, from);
                uint32_t words[4] = {r[u].x, r[u].y, r[u].z, r[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t o = 0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float x = __fmul_rn((float)(int8_t)(words[j] >> (8 * b)), rs[u]);
                        o |= (uint32_t)(scale > 0.f ? requantise(x, scale) : 0) << (8 * b);
                    }
                    words[j] = o;
                }
                if (dst >= 0)
                    *(reinterpret_cast<uint4 *>(pool + dst * pitch) + lane % LPR) =
                        make_uint4(words[0], words[1], words[2], words[3]);
            }
            if (lane == 0 && local % p.block_size == 0 && m.dst >= 0)
                scales[m.dst / p.block_size * p.hkv + h] = scale;
            if (w && m.from > i) w[i] = wv;
        }
    }
    if (w)
        for (int t = n + threadIdx.x; t < L; t += kMoveThreads) w[t] = 0.f;
}

// Strides of the weights [num_seqs, num_kv_heads, max_keys], keys contiguous.
pkv_status check_weights(const float *w, int64_t seq_stride, int64_t head_stride, int64_t max_keys, int32_t hkv,
                         const char *what) {
    PKV_CHECK_ARG((reinterpret_cast<uintptr_t>(w) & 3) == 0, PKV_ERR_INVALID_ARG, "%s: weights must be 4-byte aligned",
                  what);
    PKV_CHECK_ARG(max_keys >= 0 && max_keys < (int64_t)1 << 31, PKV_ERR_SHAPE, "%s: max_keys out of range", what);
    PKV_CHECK_ARG(head_stride >= max_keys && seq_stride >= (int64_t)(hkv - 1) * head_stride + max_keys, PKV_ERR_SHAPE,
                  "%s: rows of the weights overlap", what);
    return PKV_OK;
}

pkv_status check_compact(const int32_t *tables, int32_t max_blocks, const int32_t *seq_lens, int32_t num_seqs,
                         const int32_t *kept, int32_t budget, const float *w, int64_t seq_stride, int64_t head_stride,
                         int32_t hkv, int32_t bs, const char *what) {
    PKV_CHECK_ARG(num_seqs >= 0 && max_blocks >= 0, PKV_ERR_INVALID_ARG, "%s: negative size", what);
    PKV_CHECK_ARG(budget > 0, PKV_ERR_INVALID_ARG, "%s: budget must be positive", what);
    PKV_CHECK_ARG(bs % 16 == 0 && bs <= 256, PKV_ERR_UNSUPPORTED, "%s: block_size must be a multiple of 16 up to 256",
                  what);
    PKV_CHECK_ARG((int64_t)max_blocks * bs < (int64_t)1 << 31, PKV_ERR_SHAPE, "%s: tables cover 2^31 keys or more", what);
    PKV_CHECK_ARG((int64_t)num_seqs * hkv < (int64_t)1 << 27, PKV_ERR_UNSUPPORTED, "%s: too many rows", what);
    if (num_seqs == 0) return PKV_OK;
    PKV_CHECK_ARG(tables && seq_lens && kept, PKV_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (w) return check_weights(w, seq_stride, head_stride, (int64_t)max_blocks * bs, hkv, what);
    return PKV_OK;
}

}  // namespace

pkv_status check_cache_i8(const pkv_cache_i8 *c, const char *what);  // int8_write.cu

}  // namespace pkv

using namespace pkv;

extern "C" {

pkv_status pkv_evict_select(const float *weights, int64_t weights_seq_stride, int64_t weights_head_stride,
                            int64_t max_keys, const int32_t *seq_lens, int32_t num_seqs, int32_t num_kv_heads,
                            int32_t budget, int32_t sink, int32_t recent, int32_t *kept, int32_t *new_lens,
                            int32_t *err_word, pkv_stream stream) {
    const char *what = "pkv_evict_select";
    PKV_CHECK_ARG(num_seqs >= 0 && num_kv_heads > 0, PKV_ERR_INVALID_ARG, "%s: bad sizes", what);
    PKV_CHECK_ARG(budget > 0 && sink >= 0 && recent >= 0 && (int64_t)sink + recent <= budget, PKV_ERR_INVALID_ARG,
                  "%s: budget %d must be positive and cover sink %d + recent %d", what, budget, sink, recent);
    PKV_CHECK_ARG((int64_t)num_seqs * num_kv_heads < (int64_t)1 << 27, PKV_ERR_UNSUPPORTED, "%s: too many rows", what);
    if (num_seqs == 0) return ok();
    PKV_CHECK_ARG(weights && seq_lens && kept && new_lens, PKV_ERR_INVALID_ARG, "%s: NULL pointer", what);
    PKV_CHECK_ARG(new_lens != seq_lens, PKV_ERR_INVALID_ARG, "%s: new_lens must not be seq_lens", what);
    pkv_status st = check_weights(weights, weights_seq_stride, weights_head_stride, max_keys, num_kv_heads, what);
    if (st != PKV_OK) return st;
    SelectParams p{weights, weights_seq_stride, weights_head_stride, seq_lens, num_kv_heads, max_keys, budget, sink,
                   recent, kept, new_lens, err_word};
    st = launch_pdl(evict_select_kernel, dim3((unsigned)((int64_t)num_seqs * num_kv_heads)), dim3(kSelThreads), 0, stream,
                    p);
    return st == PKV_OK ? ok() : st;
}

pkv_status pkv_evict_compact(const pkv_cache *cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                             const int32_t *seq_lens, int32_t num_seqs, const int32_t *kept, int32_t budget,
                             float *weights, int64_t weights_seq_stride, int64_t weights_head_stride,
                             int32_t *err_word, pkv_stream stream) {
    const char *what = "pkv_evict_compact";
    pkv_status st = check_cache(cache, what);
    if (st != PKV_OK) return st;
    PKV_CHECK_ARG(cache->head_dim == 64 || cache->head_dim == 128, PKV_ERR_UNSUPPORTED,
                  "%s: head_dim must be 64 or 128 (got %d)", what, cache->head_dim);
    st = check_compact(block_tables, max_blocks_per_seq, seq_lens, num_seqs, kept, budget, weights, weights_seq_stride,
                       weights_head_stride, cache->num_kv_heads, cache->block_size, what);
    if (st != PKV_OK) return st;
    if (num_seqs == 0) return ok();
    CompactParams p{};
    p.k = cache->k;
    p.v = cache->v;
    p.tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    p.seq_lens = seq_lens;
    p.kept = kept;
    p.budget = budget;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.hkv = cache->num_kv_heads;
    p.w = weights;
    p.seq_stride = weights_seq_stride;
    p.head_stride = weights_head_stride;
    p.chunk = kChunk;
    p.err = err_word;
    const dim3 grid((unsigned)((int64_t)num_seqs * cache->num_kv_heads * 2));
    st = cache->head_dim == 64 ? launch_pdl(evict_compact_kernel<128>, grid, dim3(kMoveThreads), 0, stream, p)
                               : launch_pdl(evict_compact_kernel<256>, grid, dim3(kMoveThreads), 0, stream, p);
    return st == PKV_OK ? ok() : st;
}

pkv_status pkv_evict_compact_int8(const pkv_cache_i8 *cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                  const int32_t *seq_lens, int32_t num_seqs, const int32_t *kept, int32_t budget,
                                  float *weights, int64_t weights_seq_stride, int64_t weights_head_stride,
                                  int32_t *err_word, pkv_stream stream) {
    const char *what = "pkv_evict_compact_int8";
    pkv_status st = check_cache_i8(cache, what);
    if (st != PKV_OK) return st;
    PKV_CHECK_ARG(cache->head_dim == 128, PKV_ERR_UNSUPPORTED, "%s: head_dim must be 128", what);
    st = check_compact(block_tables, max_blocks_per_seq, seq_lens, num_seqs, kept, budget, weights, weights_seq_stride,
                       weights_head_stride, cache->num_kv_heads, cache->block_size, what);
    if (st != PKV_OK) return st;
    if (num_seqs == 0) return ok();
    CompactParams p{};
    p.k = cache->k;
    p.v = cache->v;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    p.seq_lens = seq_lens;
    p.kept = kept;
    p.budget = budget;
    p.num_blocks = cache->num_blocks;
    p.block_size = cache->block_size;
    p.hkv = cache->num_kv_heads;
    p.w = weights;
    p.seq_stride = weights_seq_stride;
    p.head_stride = weights_head_stride;
    p.chunk = kChunk / cache->block_size * cache->block_size;
    p.err = err_word;
    const dim3 grid((unsigned)((int64_t)num_seqs * cache->num_kv_heads * 2));
    st = launch_pdl(evict_compact_i8_kernel, grid, dim3(kMoveThreads), 0, stream, p);
    return st == PKV_OK ? ok() : st;
}

}  // extern "C"
