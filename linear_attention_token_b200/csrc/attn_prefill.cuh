// What the two gdn_attn_prefill kernels share: the call's parameters, the sequences' tokens, what
// a query sees, and the scores' scaling.
#pragma once

#include <math.h>

#include "attn_math.cuh"
#include "paged_kv.cuh"

namespace gdn {

struct AttnPrefillParams {
    PagedView cache;
    const void *q;
    void *out;
    float *lse;
    const int32_t *cu, *pos0, *prefix;
    long long T_total, T_seq;              // T_seq: tokens per sequence when cu is null
    int N, H_q, G, window;
    bool heads_first;                      // order of the CTAs
    int pack_shift;                        // rows of a tile: token r >> pack_shift, head the rest
    Scoring score;
    float near_at, nearer_at;              // largest |score / cap| of the cap's two polynomials
    DeviceError *err;
    uint32_t budget;
    long long blocks;                      // (block, head) pairs, as prefill_shape counts them
    // A long context with few blocks: `splits` CTAs share a block's tokens, and their parts (of
    // part_rows rows, m and l, and unnormalised outputs) are joined by attn_prefill_join_kernel.
    int splits;                            // 1: none
    struct SplitBlock *split_blocks;       // [blocks x heads]
    float2 *part_ml;                       // [blocks x heads, splits, part_rows]
    float *part_o;                         // [.., d]
};

// What a split block's first CTA leaves for the join.  Row r of the block is token
// (row0 + r) / pack of the sequence and head h0 + (row0 + r) % pack.
struct SplitBlock {
    long long first;
    int len, row0, pack, h0;
    int parts;                             // CTAs that took a share (0 or 1: nothing to join)
    int pad;
};

// How the two kernels cut a call (their CTAs' query rows and K / V tiles).
constexpr int kPrefillTile = 128, kPrefillRows = 2 * kPrefillTile;             // bf16
constexpr int kF32Rows = 64, kF32Keys = 64;                                    // fp32

// Least K / V tiles that are worth a CTA of their own (16 rows behind 2048 tokens: 18.8 us with 3, 19.6
// with 4, 26 with 8, 35 in one piece; 300 x 2 x 8 rows behind 1024: 24, 26, 28, 28).
constexpr int kSplitTiles = 3;

// CTAs that share a block's `tiles`, and the share of CTA s: tiles [from, to).
__device__ __forceinline__ int split_parts(int tiles, int splits) {
    return max(1, min(splits, tiles / kSplitTiles));
}
__device__ __forceinline__ void split_range(int tiles, int parts, int s, int &from, int &to) {
    from = (int)((long long)tiles * s / parts);
    to = (int)((long long)tiles * (s + 1) / parts);
}
// A sequence of the call: the row of its first token in q and out, its tokens, those cached before
// them, and its prefix.
struct Sequence {
    long long first;
    int len, start, pre;
};
// Sequence n, inside the call's T_total tokens whatever the offsets say.
__device__ __forceinline__ Sequence sequence_of(const AttnPrefillParams &p, int n) {
    Sequence s;
    s.start = p.pos0 ? __ldg(p.pos0 + n) : 0;
    s.pre = p.prefix ? __ldg(p.prefix + n) : 0;
    if (!p.cu) {
        s.first = n * p.T_seq;
        s.len = (int)p.T_seq;
        return s;
    }
    s.first = __ldg(p.cu + n);
    const long long end = min((long long)__ldg(p.cu + n + 1), p.T_total);
    s.len = s.first >= 0 && end > s.first ? (int)(end - s.first) : 0;
    return s;
}

// What the queries of a sequence see: query i sees the tokens [lo(i), hi(i)), both growing with i and
// inside [0, e].  e may be the last 32-bit position but 15, so a tile's end may not fit an int: what
// follows compares distances from a tile's first token, never its end.
struct Sight {
    long long start;
    int e, pre, window;
    __device__ __forceinline__ Sight(const AttnPrefillParams &p, const Sequence &s) {
        start = s.start;
        e = (int)min(max(start + s.len, 0LL), cache_capacity(p.cache));
        pre = max(min(s.pre, e), 0);
        window = p.window;
    }
    __device__ __forceinline__ int hi(int i) const {
        return (int)max(min(start + i + 1, (long long)e), (long long)pre);
    }
    __device__ __forceinline__ int lo(int i) const {
        return window > 0 ? (int)min(max(start + i - window + 1, 0LL), (long long)e) : 0;
    }
};

// Block x of the call: its sequence (n, s) and its number b there.  blocks_of(len) is a sequence's
// number of blocks; they are numbered from the last one back, since a sequence's last blocks see
// the most tokens and should start first.  All THREADS threads call it, and it ends with a barrier;
// false when x is past the last block.
template <int THREADS, class F>
__device__ __forceinline__ bool find_block(const AttnPrefillParams &p, F &&blocks_of, long long x,
                                           int &n, int &b, Sequence &s) {
    __shared__ int sums[THREADS / 32], found[2];
    __shared__ Sequence sequence;
    if (!p.cu) {
        const long long at = blocks_of(p.T_seq) * p.N - 1 - x;
        b = (int)(at / p.N);               // the last blocks of all sequences first
        n = (int)(at % p.N);
        if (at >= 0) s = sequence_of(p, n);
        __syncthreads();
        return at >= 0;
    }
    // thread t counts the blocks of sequences [t per, t per + per); all that is needed of a
    // sequence is loaded at once, so the search costs one trip to memory
    const int tid = threadIdx.x, per = (p.N + THREADS - 1) / THREADS;
    const int n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
    const int lane = tid & 31, warp = tid >> 5;
    int mine = 0;
    s = Sequence{0, 0, 0, 0};
    for (int i = n0; i < n1; ++i) {
        s = sequence_of(p, i);
        mine += (int)blocks_of(s.len);
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sums[warp] = inc;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int before = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const int at = (int)(total - 1 - x);
    if (at >= before && at < before + mine) {
        int left = at - before, i = n0;
        if (per > 1)
            for (;; ++i) {
                s = sequence_of(p, i);
                const int nb = (int)blocks_of(s.len);
                if (left < nb) break;
                left -= nb;
            }
        found[0] = i;
        found[1] = left;
        sequence = s;
    }
    __syncthreads();
    n = found[0];
    b = found[1];
    s = sequence;
    return n >= 0;
}

}  // namespace gdn
