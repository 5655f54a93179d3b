// gdn_attn_decode and gdn_qsa_attn_decode (include/attn.h): attention of the newest tokens of
// every sequence over the paged cache, whole or by lists.
//
//   out = sum_t e^{x_t - m} v_t / sum_t e^{x_t - m},  m = max_t x_t,  x_t = cap(scale q . k_t)
//
// in one pass over the keys with a running m and sum; parts of a sequence that different CTAs
// (or warps) ran are joined by out = sum_i e^{m_i - m} O_i / sum_i e^{m_i - m} l_i.
//
// Every visible key and value is read once for all the query rows that share it (the heads of
// its group, and the drafted tokens when no lists are given), so the calls are bound by HBM:
// per key and head 4 d bytes (bf16) against at most 4 d flops per query row.
//
//  - Work split.  A unit is one (sequence, key head[, row block][, drafted token]); its keys are
//    cut into steps of 64.  The steps of all units form one line, and each CTA takes an equal
//    stretch of it, wherever units begin and end: ragged lengths cost nothing, one long
//    sequence uses every SM, and no length is needed on the host (a captured graph stays valid
//    as sequences grow).  A unit that lies in one CTA is finished there; the parts of the
//    others go to the workspace (at most two per CTA), and attn_join_kernel, launched beside this
//    one, joins them.  (The last CTA of a unit joining in this kernel was slower on every size: one
//    CTA's fences, atomics and cold code at the end cost more than a second grid.)
//    Short calls of few units take a cluster of CTAs to a unit instead, which join their parts in
//    shared memory and need no second grid (cluster_for); drafts of many rows behind a short table
//    the prompt kernel (many_rows).
//  - bf16: a warp owns 16 query rows as one mma.sync m16n8k16 row tile.  With few rows the
//    product is far from the tensor pipe's limit, so what counts is that loads never pause:
//    each team of warps (1, 2 or 4 by the number of rows) streams its own keys through a
//    private ring of cp.async stages and waits for nobody else.
//  - fp32: the same skeleton with fp32 FMAs (one product of operands of fewer bits would not hold 1e-4).
//
// Measured (cache bytes over time; a plain copy moves 6.45 TB/s): 8 sequences of 262,144 tokens x 2 heads
// bf16 320 us, 6.7 TB/s; 64 ragged ones of 2000 to 16,384 tokens x 8 heads, two drafted tokens each, 356 us,
// 6.6 TB/s; one of 262,144 tokens x 2 heads 53 us, 5.1 TB/s; d = 64, 64 x 8192 tokens x 8 heads 183 us, 5.9
// TB/s. 64 x 16,384 tokens x 8 heads with a window of 1024: 51 us, 5.2 TB/s, of 4096: 164, 6.5. Lists of
// 2048 tokens for 32 x 4 drafted queries: 55 us, 4.9 TB/s, in fp32 150, 3.7 TB/s, d = 64 40, 3.4; 4 x 1024
// tokens: 6.6 us, mostly the launch and the chain position -> page table -> keys.
// Where it is not the bytes: bf16, 17 to 32 rows (64 x 4096 x 2 heads, 32 rows: 60 us, 4.5 TB/s; 16 rows 54): two warps
// read each tile whole by ldmatrix, 255 registers leave 8 warps an SM, and 61% of the cycles have none
// that can issue (tensor pipe 32%). fp32, the same tokens: 84 us with one row a head, 6.4 TB/s; 99 with four;
// 129 with eight, 17 TFLOP/s: the ring of d = 128 leaves one CTA of four warps an SM, and 69% of the
// cycles have none that can issue (FMA pipe 29%).
#include <math.h>
#include <stdint.h>

#include "attn_math.cuh"
#include "device_once.h"
#include "paged_kv.cuh"
#include "sm100.cuh"

namespace gdn {
// CTAs that share a block of a dense call of the prompt kernel when its table holds a long context
int attn_prefill_splits(const gdn_paged_kv &kv, int N, long long T_total, int H_q, int sms);

using sm100::cluster_rank;
using sm100::cluster_size;
using sm100::cluster_sync;
using sm100::ld_cluster2;
using sm100::ld_cluster4;
using sm100::map_to_rank;

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr int kMostCluster = 16;
constexpr int kLoad = 16;                  // keys one warp loads per step
constexpr int kStep = kWarps * kLoad;      // keys per step of a CTA
// Growth of a row's maximum (base 2) that its sums may lag: until then the old one serves, and
// nothing is rescaled. The largest weight is then no longer an exact 1 of bf16, which costs accuracy
// (2 x 262,144 tokens, against 64 bits, relative: 0 -> .0021, 2 -> .0022, 8 -> .0023), while the
// time is 56.1 / 55.6 / 55.2 us on lists of four drafts and the same everywhere else.
constexpr float kLazy = 2.f;

// What the CTA in which a unit begins leaves for the join.
struct JoinRecord {
    int n, sub;                            // sequence; unit within the sequence
    int parts;                             // CTAs c .. c + parts - 1 hold a part (0: nothing to join)
    int place;                             // 2 c + where CTA c's own part is (later ones: slot 0)
};

struct DecodeParams {
    PagedView cache;
    const void *q;
    const int32_t *q_pos, *list;
    void *out;
    float *lse;
    float *part_o;                         // [grid, 2, rows, D]
    float2 *part_ml;                       // [grid, 2, rows]
    JoinRecord *rec;                       // [grid]: by unit while there are no more than that, else by CTA
    bool by_unit;
    int N, T, H_q, G;                      // G = H_q / H_kv
    int rows, row_blocks;                  // query rows of a unit (before blocking), blocks
    int units_per_seq;
    int list_len, recent, window;
    Scoring score;
};

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes global -> shared; reads nothing and writes zeros when !live
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;"
                 ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// --------------------------------------------------------------------- where the work is
// Keys that unit (n, sub) walks: dense, tokens [lo, hi) with lo on a step; lists, positions
// of list (padded to a step) and newest tokens.
struct Span {
    long long lo;                          // dense: first token of step 0
    int steps;
};

template <bool LIST>
__device__ __forceinline__ Span span_of(const DecodeParams &p, int n) {
    Span s;
    if (LIST) {
        s.lo = 0;
        s.steps = (p.list_len + kStep - 1) / kStep + (p.recent + kStep - 1) / kStep;
    } else {
        const long long pos = __ldg(p.q_pos + n);
        long long hi = pos + p.T;                                // one past the last query
        const long long cap = cache_capacity(p.cache);
        hi = hi < cap ? hi : cap;
        s.lo = p.window > 0 && pos - p.window + 1 > 0 ? (pos - p.window + 1) / kStep * kStep : 0;
        s.steps = hi > s.lo ? (int)((hi - s.lo + kStep - 1) / kStep) : 0;
    }
    if (s.steps < 1) s.steps = 1;          // a unit that sees nothing still writes its zeros
    return s;
}

struct Unit {
    int n, sub;                            // sequence, unit within it
    int h, rb, j;                          // key head, row block, drafted token (lists)
};
template <bool LIST>
__device__ __forceinline__ Unit unit_of(const DecodeParams &p, int n, int sub) {
    Unit u;
    u.n = n;
    u.sub = sub;
    u.rb = sub % p.row_blocks;
    u.h = sub / p.row_blocks % p.cache.H_kv;
    u.j = LIST ? sub / (p.row_blocks * p.cache.H_kv) : 0;
    return u;
}
// (token, head) of row r of a unit
template <bool LIST>
__device__ __forceinline__ size_t row_head(const DecodeParams &p, const Unit &u, int r) {
    const int j = LIST ? u.j : r / p.G, g = LIST ? r : r % p.G;
    return ((size_t)u.n * p.T + j) * p.H_q + (size_t)u.h * p.G + g;
}

// ------------------------------------------------------------------------------- loading
// Token of key `key` of warp `sub`'s share of a step, or -1: not seen by any query of the
// unit.  (What nobody sees is not read: it may hold anything.)
template <bool LIST>
__device__ __forceinline__ int token_at(const DecodeParams &p, const Unit &u, const Span &sp,
                                        long long pos, int step, int sub, int key) {
    const int i = step * kStep + sub * kLoad + key;
    if (LIST) {
        const int list_pad = (p.list_len + kStep - 1) / kStep * kStep;
        const long long at = pos + u.j;
        if (i < list_pad) {
            if (i >= p.list_len) return -1;
            const int t = __ldg(p.list + ((size_t)u.n * p.T + u.j) * p.list_len + i);
            return t <= at - p.recent ? t : -1;
        }
        const long long t = at - p.recent + 1 + (i - list_pad);
        return i - list_pad < p.recent && t >= 0 && t <= INT32_MAX ? (int)t : -1;
    }
    const long long t = sp.lo + i;
    const bool seen = t < pos + p.T && (p.window <= 0 || t > pos - p.window) && t <= INT32_MAX;
    return seen ? (int)t : -1;
}

// One warp's keys of one step into its rows of a stage (rows of D elements, 16-byte
// chunk c of row r at c ^ (r & 7)), keys at kdst, values at vdst.  Lane l < 16 holds the cache
// row of key l; absent keys (-1) are zero-filled, so nothing a dead row holds reaches a product.
template <typename E, int D>
__device__ __forceinline__ void load_keys(const DecodeParams &p, int h, int row, uint32_t kdst,
                                          uint32_t vdst) {
    constexpr int CH = D * (int)sizeof(E) / 16, RPI = 32 / CH, ITER = kLoad / RPI;
    const int lane = threadIdx.x & 31, c = lane % CH;
    const size_t pitch = (size_t)p.cache.H_kv * D * sizeof(E);
    const size_t off = (size_t)h * D * sizeof(E) + (size_t)c * 16;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
        const int r = lane / CH + i * RPI;
        const int at = __shfl_sync(0xffffffffu, row, r);
        const size_t src = (size_t)(at < 0 ? 0 : at) * pitch + off;
        const uint32_t d = (uint32_t)(r * CH + (c ^ (r & 7))) * 16;
        cp_async16(kdst + d, p.cache.k + src, at >= 0);
        cp_async16(vdst + d, p.cache.v + src, at >= 0);
    }
}

// ------------------------------------------------------------------- bf16: tensor cores
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A warp's 16 query rows against the keys of its team.  Lane (g = lane / 4, c = lane % 4) holds
// rows g and g + 8: scores of keys 8 i + 2 c, + 1; outputs of dims 8 i + 2 c, + 1.
template <int D, int TEAM, bool LIST>
struct TensorRows {
    using E = __nv_bfloat16;
    static constexpr int kTeam = TEAM, kRows = 16 * TEAM;        // rows of a unit's block
    static constexpr int kTileKeys = kLoad * TEAM;
    uint32_t q[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];
    int first[2], last[2];                 // tokens row g / g + 8 may see (dense)

    __device__ void begin(const DecodeParams &p, const Unit &u, long long pos, float *) {
        const int lane = threadIdx.x & 31, wt = (threadIdx.x >> 5) % TEAM;
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = u.rb * kRows + wt * 16 + g + 8 * e;
            const bool live = r < p.rows;
            const E *src = static_cast<const E *>(p.q) + row_head<LIST>(p, u, live ? r : 0) * D + 2 * c;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                q[k][e] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k)) : 0u;
                q[k][e + 2] = live ? __ldg(reinterpret_cast<const uint32_t *>(src + 16 * k + 8)) : 0u;
            }
            m[e] = -INFINITY;
            l[e] = 0.f;
            const long long at = pos + (LIST || !live ? 0 : r / p.G);
            last[e] = LIST ? INT32_MAX : (int)(at < INT32_MAX ? at : INT32_MAX);
            first[e] = LIST || p.window <= 0 ? INT32_MIN
                       : (int)(at - p.window + 1 > INT32_MIN ? at - p.window + 1 : INT32_MIN);
        }
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }

    // kt, vt: the team's tile of kTileKeys rows; token0: token of its key 0 (dense)
    __device__ __forceinline__ void tile(const DecodeParams &p, uint32_t kt, uint32_t vt,
                                         uint64_t present, long long token0, float *) {
        constexpr int NT = kTileKeys / 8;
        const int lane = threadIdx.x & 31, c = lane & 3;
        float s[NT][4];
        const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            const int r = 16 * i + kr;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t b[4];
                ldsm4(kt + (uint32_t)(r * (D / 8) + ((2 * k + kc) ^ (r & 7))) * 16, b);
                mma16816(s[2 * i], q[k], b[0], b[1]);
                mma16816(s[2 * i + 1], q[k], b[2], b[3]);
            }
        }
        score2<5>(reinterpret_cast<float(&)[NT * 4]>(s), p.score);
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = 8 * i + 2 * c + (e & 1);
                bool live = (present >> key) & 1;
                if (!LIST) {
                    const int t = (int)(token0 + key);
                    live = live && t <= last[e >> 1] && t >= first[e >> 1];
                }
                s[i][e] = live ? s[i][e] : -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], s[i][e]);
            }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kLazy || mx[1] > m[1] + kLazy)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                mx[e] = fmaxf(mx[e], m[e]);
                const float f = mx[e] == -INFINITY ? 1.f : ex2(m[e] - mx[e]);       // 0 while m is -inf
                m[e] = mx[e];
                l[e] *= f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) { o[i][2 * e] *= f; o[i][2 * e + 1] *= f; }
            }
        }
        const float shift[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
        // rounded to bf16 for the product (each weight is off by half a step, 2^-8 of itself, at
        // most; over many keys the errors average out below the output's own rounding); the sum
        // takes the unrounded weights, so lse has no part in it
        uint32_t w[NT / 2][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float a = ex2(s[i][2 * e] - shift[e]), b = ex2(s[i][2 * e + 1] - shift[e]);
                l[e] += a + b;
                w[i >> 1][(i & 1) * 2 + e] = pack2(a, b);
            }
        const int vr = (lane & 7) + ((lane >> 3) & 1) * 8, vc = lane >> 4;
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {
            const int r = 16 * k + vr;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t b[4];
                ldsm4t(vt + (uint32_t)(r * (D / 8) + ((2 * i + vc) ^ (r & 7))) * 16, b);
                mma16816(o[2 * i], w[k], b[0], b[1]);
                mma16816(o[2 * i + 1], w[k], b[2], b[3]);
            }
        }
    }

    // this warp's part: rows at so[kRows][D], maxima and sums at sml[kRows]
    __device__ void put(float *so, float2 *sml) {
        const int lane = threadIdx.x & 31, wt = (threadIdx.x >> 5) % TEAM;
        const int g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = wt * 16 + g + 8 * e;
            float sum = l[e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (c == 0) sml[r] = make_float2(m[e], sum);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(so + r * D + 8 * i + 2 * c) =
                    make_float2(o[i][2 * e], o[i][2 * e + 1]);
        }
    }
};

// --------------------------------------------------------------------- fp32: CUDA cores
// A warp's keys against R query rows held in shared memory.  Scores: kLanes lanes a key, each some of
// the dims; weights go through shared memory; outputs: lane owns D / 32 dims of every row.
template <int D, int R, bool LIST>
struct FmaRows {
    using E = float;
    static constexpr int kTeam = 1, kRows = R, kTileKeys = kLoad, kV = D / 32;
    static constexpr int kLanes = 32 / kLoad;                  // lanes that share a key
    float2 o[R][kV / 2];
    float m[R], l[R];
    int first[R], last[R];                 // tokens a row may see (dense)

    // shared: q [R][D], then per warp weights [R][kLoad]
    __device__ void begin(const DecodeParams &p, const Unit &u, long long pos, float *shared) {
        for (int i = threadIdx.x; i < R * D; i += kThreads) {
            const int r = u.rb * R + i / D;
            shared[i] = r < p.rows ? __ldg(static_cast<const float *>(p.q) +
                                           row_head<LIST>(p, u, r) * D + i % D) : 0.f;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const long long at = pos + (LIST ? 0 : (u.rb * R + r) / p.G);
            last[r] = LIST ? INT32_MAX : (int)min(at, (long long)INT32_MAX);
            first[r] = LIST || p.window <= 0 ? INT32_MIN : (int)max(at - p.window + 1, (long long)INT32_MIN);
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < kV / 2; ++e) o[r][e] = make_float2(0.f, 0.f);
        }
        __syncthreads();
    }

    __device__ __forceinline__ void tile(const DecodeParams &p, uint32_t kt, uint32_t vt,
                                         uint64_t present, long long token0, float *shared) {
        constexpr int CH = D / 4;
        const int lane = threadIdx.x & 31, key = lane / kLanes, part = lane % kLanes;
        float2 s2[R];
#pragma unroll
        for (int r = 0; r < R; ++r) s2[r] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < CH / kLanes; ++c) {
            const int ch = kLanes * c + part;                   // a key's lanes read neighbours
            float4 k;
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(k.x), "=f"(k.y), "=f"(k.z), "=f"(k.w)
                         : "r"(kt + (uint32_t)(key * CH + (ch ^ (key & 7))) * 16) : "memory");
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 q = *reinterpret_cast<const float4 *>(shared + r * D + ch * 4);
                s2[r] = fma2(make_float2(q.x, q.y), make_float2(k.x, k.y), s2[r]);
                s2[r] = fma2(make_float2(q.z, q.w), make_float2(k.z, k.w), s2[r]);
            }
        }
        float *w = shared + R * D + (threadIdx.x >> 5) * R * kLoad;
        float s[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            s[r] = s2[r].x + s2[r].y;
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) s[r] += __shfl_xor_sync(0xffffffffu, s[r], d);
        }
        score2<7>(s, p.score);
        const int t = (int)(token0 + key);
        const bool there = (present >> key) & 1;
        bool grow = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (!there || (!LIST && (t > last[r] || t < first[r]))) s[r] = -INFINITY;
            grow = grow || s[r] > m[r] + kLazy;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mx = s[r];
#pragma unroll
                for (int d = kLanes; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                mx = fmaxf(mx, m[r]);
                const float f = mx == -INFINITY ? 1.f : ex2(m[r] - mx);             // 0 while m is -inf
                m[r] = mx;
                l[r] *= f;
#pragma unroll
                for (int v = 0; v < kV / 2; ++v) o[r][v] = make_float2(o[r][v].x * f, o[r][v].y * f);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float e = ex2(s[r] - (m[r] == -INFINITY ? 0.f : m[r]));
            if (part == 0) {
                l[r] += e;
                w[r * kLoad + key] = e;
            }
        }
        __syncwarp();
#pragma unroll
        for (int k0 = 0; k0 < kLoad; k0 += 4) {
            float2 v[4][kV / 2];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t at = vt + (uint32_t)((k0 + k) * CH + ((lane * kV >> 2) ^ ((k0 + k) & 7))) * 16;
                if constexpr (kV == 4)
                    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(v[k][0].x), "=f"(v[k][0].y), "=f"(v[k][1].x), "=f"(v[k][1].y) : "r"(at) : "memory");
                else
                    asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];"
                                 : "=f"(v[k][0].x), "=f"(v[k][0].y) : "r"(at + (lane & 1) * 8) : "memory");
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 x = *reinterpret_cast<const float4 *>(w + r * kLoad + k0);
#pragma unroll
                for (int e = 0; e < kV / 2; ++e) {
                    o[r][e] = fma2(make_float2(x.x, x.x), v[0][e], o[r][e]);
                    o[r][e] = fma2(make_float2(x.y, x.y), v[1][e], o[r][e]);
                    o[r][e] = fma2(make_float2(x.z, x.z), v[2][e], o[r][e]);
                    o[r][e] = fma2(make_float2(x.w, x.w), v[3][e], o[r][e]);
                }
            }
        }
        __syncwarp();
    }

    __device__ void put(float *so, float2 *sml) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = warp_sum(l[r]);
            if (lane == 0) sml[r] = make_float2(m[r], sum);
#pragma unroll
            for (int e = 0; e < kV / 2; ++e)
                *reinterpret_cast<float2 *>(so + r * D + lane * kV + 2 * e) = o[r][e];
        }
    }
};

// -------------------------------------------------------------------------------- kernel
template <class ROWS, int D>
struct Layout {
    static constexpr int kTeams = kWarps / ROWS::kTeam;
    static constexpr int kRowBytes = D * (int)sizeof(typename ROWS::E);
    static constexpr int kStageBytes = kStep * kRowBytes;              // K or V of one step
    static constexpr int kRing = kStages * 2 * kStageBytes;
    // the join of the CTA's teams reuses the ring
    static constexpr int kJoin = (kTeams + 1) * ROWS::kRows * (D + 2) * 4;    // (+ 1: the CTA's part, in a cluster)
    static constexpr int kExtra = sizeof(typename ROWS::E) == 4 ? (ROWS::kRows * D + kWarps * ROWS::kRows * kLoad) * 4 : 0;
    static constexpr int kMask = kStages * kWarps * 4;
    static constexpr int kBody = kRing > kJoin ? kRing : kJoin;
    static constexpr int kSmem = kBody + kExtra + kMask + 64;
};

template <int TEAM> __device__ __forceinline__ void team_sync() {
    if (TEAM == 1) __syncwarp();
    else if (TEAM == kWarps) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)(threadIdx.x >> 5) / TEAM), "n"(32 * TEAM) : "memory");
}

// First step of CTA c's stretch when G CTAs share W steps, and the CTA that runs step x.
__device__ __forceinline__ long long stretch(long long W, int G, int c) {
    const unsigned long long x = (unsigned long long)W * c;
    return x >> 32 ? (long long)(x / G) : (long long)((uint32_t)x / (uint32_t)G);
}
__device__ __forceinline__ int cta_of(long long W, int G, long long x) {
    const unsigned long long y = (unsigned long long)(x + 1) * G + W - 1;
    return (y >> 32 ? (int)(y / W) : (int)((uint32_t)y / (uint32_t)W)) - 1;
}

// Four output columns of one row: maximum m, sum l, columns o.
struct Sums {
    float m, l;
    float4 o;
};
// The sums of up to N parts: their m and l, and their columns, are loaded together, and the weights
// e^{m_i - m} do not depend on one another.
template <int N, class ML, class O>
__device__ __forceinline__ Sums sum_parts(int count, ML &&ml_of, O &&o_of) {
    float2 ml[N];
    float4 o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        ml[i] = i < count ? ml_of(i) : make_float2(-INFINITY, 0.f);
        o[i] = i < count ? o_of(i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    Sums s;
    s.m = ml[0].x;
#pragma unroll
    for (int i = 1; i < N; ++i) s.m = fmaxf(s.m, ml[i].x);
    const float shift = s.m == -INFINITY ? 0.f : s.m;
    s.l = 0.f;
    s.o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float f = ex2(ml[i].x - shift);
        s.l = fmaf(ml[i].y, f, s.l);
        s.o.x = fmaf(o[i].x, f, s.o.x);
        s.o.y = fmaf(o[i].y, f, s.o.y);
        s.o.z = fmaf(o[i].z, f, s.o.z);
        s.o.w = fmaf(o[i].w, f, s.o.w);
    }
    return s;
}

template <typename E> __device__ __forceinline__ void store4(void *p, size_t i, float4 x);
template <> __device__ __forceinline__ void store4<float>(void *p, size_t i, float4 x) {
    *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) = x;
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(void *p, size_t i, float4 x) {
    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p) + i) = make_uint2(pack2(x.x, x.y), pack2(x.z, x.w));
}

template <typename E, int D, bool LIST>
__device__ __forceinline__ void finish(const DecodeParams &p, const Unit &u, int row, int c, const Sums &s) {
    const size_t rh = row_head<LIST>(p, u, row);
    const float inv = s.l > 0.f ? 1.f / s.l : 0.f;
    store4<E>(p.out, rh * D + c, make_float4(s.o.x * inv, s.o.y * inv, s.o.z * inv, s.o.w * inv));
    if (c == 0 && p.lse) p.lse[rh] = s.l > 0.f ? (s.m + log2f(s.l)) * kLn2 : -INFINITY;
}

// CLUSTER: a cluster of CTAs takes a unit, and they join their parts in shared memory.
template <class ROWS, int D, bool LIST, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
attn_decode_kernel(const __grid_constant__ DecodeParams p) {
    using E = typename ROWS::E;
    using L = Layout<ROWS, D>;
    constexpr int TEAM = ROWS::kTeam;
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ long long sums[kWarps], found[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *extra = reinterpret_cast<float *>(sm + L::kBody);
    uint32_t *masks = reinterpret_cast<uint32_t *>(sm + L::kBody + L::kExtra);   // [stage][warp]

    // all steps, and where this CTA's stretch begins
    const int cta = blockIdx.x;
    if (!CLUSTER) {
        pdl_trigger();
        if (tid == 0 && !p.by_unit) p.rec[cta].parts = 0;
    }
    long long W = 0, begin = 0, end;
    int G = 0, n, sub, step;
    Span sp;
    if (CLUSTER) {                         // a unit's steps from `step` on
        const int size = cluster_size(), rank = cluster_rank(), unit = cta / size;
        n = unit / p.units_per_seq;
        sub = unit - n * p.units_per_seq;
        sp = span_of<LIST>(p, n);
        step = (int)((long long)sp.steps * rank / size);
        end = (long long)sp.steps * (rank + 1) / size - step;    // may be 0: an empty part
    } else if (LIST) {                     // every unit has the same steps
        sp = span_of<LIST>(p, 0);
        W = (long long)p.N * p.units_per_seq * sp.steps;
        G = (int)(W < (long long)gridDim.x ? W : gridDim.x);
        if (cta >= G) return;
        begin = stretch(W, G, cta);
        const long long unit = begin / sp.steps;
        step = (int)(begin - unit * sp.steps);
        n = (int)(unit / p.units_per_seq);
        sub = (int)(unit - (long long)n * p.units_per_seq);
    } else {                               // thread t sums sequences [t per, t per + per)
        const int per = (p.N + kThreads - 1) / kThreads;
        const int n0 = min(p.N, tid * per), n1 = min(p.N, n0 + per);
        long long mine = 0;
        for (int i = n0; i < n1; ++i) mine += (long long)span_of<LIST>(p, i).steps * p.units_per_seq;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) sums[warp] = upto;
        __syncthreads();
        W = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) upto += sums[w];
            W += sums[w];
        }
        G = (int)(W < (long long)gridDim.x ? W : gridDim.x);
        if (cta >= G) return;
        begin = stretch(W, G, cta);
        if (upto - mine <= begin && begin < upto) {
            long long at = upto - mine;
            for (int i = n0; i < n1; ++i) {
                const long long x = (long long)span_of<LIST>(p, i).steps * p.units_per_seq;
                if (begin < at + x) { found[0] = i; found[1] = begin - at; break; }
                at += x;
            }
        }
        __syncthreads();
        n = (int)found[0];
        sp = span_of<LIST>(p, n);
        sub = (int)(found[1] / sp.steps);
        step = (int)(found[1] - (long long)sub * sp.steps);
    }
    if (!CLUSTER) end = stretch(W, G, cta + 1);

    ROWS rows;
    const int team = warp / TEAM;
    const uint32_t ring = smem_addr(sm);
    for (long long at = begin; CLUSTER || at < end;) {
        const Unit u = unit_of<LIST>(p, n, sub);
        const long long pos = __ldg(p.q_pos + n);
        const int count = (int)min((long long)(sp.steps - step), end - at);
        // tokens are looked up two steps, cache rows one step before their loads go out, so that
        // the chain list -> page table -> key never stalls a step
        auto token = [&](int i) {
            return i < count ? token_at<LIST>(p, u, sp, pos, step + i, warp, lane % kLoad) : -1;
        };
        int row = cache_row(p.cache, n, token(0)), t_ahead = token(1);
        auto load = [&](int i) {
            const int row_ahead = cache_row(p.cache, n, t_ahead);
            t_ahead = token(i + 2);
            if (i < count) {
                const int st = i % kStages;
                const uint32_t dst = ring + st * 2 * L::kStageBytes + warp * kLoad * L::kRowBytes;
                load_keys<E, D>(p, u.h, row, dst, dst + L::kStageBytes);
                const uint32_t present = __ballot_sync(0xffffffffu, row >= 0) & ((1u << kLoad) - 1);
                if (lane == 0) masks[st * kWarps + warp] = present;
            }
            cp_commit();
            row = row_ahead;
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) load(i);
        rows.begin(p, u, pos, extra);
        for (int i = 0; i < count; ++i) {
            cp_wait<kStages - 2>();
            team_sync<TEAM>();             // the tile is there, and the slot of tile i - 1 is free
            load(i + kStages - 1);
            const int st = i % kStages;
            uint64_t present = 0;
#pragma unroll
            for (int w = 0; w < TEAM; ++w)
                present |= (uint64_t)masks[st * kWarps + team * TEAM + w] << (16 * w);
            const uint32_t kt = ring + st * 2 * L::kStageBytes + team * ROWS::kTileKeys * L::kRowBytes;
            rows.tile(p, kt, kt + L::kStageBytes, present,
                      sp.lo + (long long)(step + i) * kStep + team * ROWS::kTileKeys, extra);
        }
        cp_wait<0>();
        __syncthreads();                   // the ring is free: join the teams in it
        float *so = reinterpret_cast<float *>(sm);
        float2 *sml = reinterpret_cast<float2 *>(so + L::kTeams * ROWS::kRows * D);
        rows.put(so + team * ROWS::kRows * D, sml + team * ROWS::kRows);
        __syncthreads();
        if constexpr (CLUSTER) {
            // this CTA's part [rows][D], then m and l, behind the teams' ones; each CTA joins some rows
            constexpr int R = ROWS::kRows;
            float *po = so + L::kTeams * R * (D + 2);
            float2 *pml = reinterpret_cast<float2 *>(po + R * D);
            const int live_rows = min(R, p.rows - u.rb * R);
            for (int i = tid; i < live_rows * (D / 4); i += kThreads) {
                const int r = i / (D / 4), c = 4 * (i % (D / 4));
                const Sums s = sum_parts<L::kTeams>(
                    L::kTeams, [&](int t) { return sml[t * R + r]; },
                    [&](int t) { return *reinterpret_cast<const float4 *>(so + (t * R + r) * D + c); });
                *reinterpret_cast<float4 *>(po + r * D + c) = s.o;
                if (c == 0) pml[r] = make_float2(s.m, s.l);
            }
            __syncwarp();
            cluster_sync();
            const int size = cluster_size(), c = 4 * (tid % (D / 4));
            for (int r = (int)cluster_rank() + size * (tid / (D / 4)); r < live_rows; r += size * (kThreads / (D / 4))) {
                const Sums s = sum_parts<kMostCluster>(
                    size, [&](int i) { return ld_cluster2(map_to_rank(pml + r, i)); },
                    [&](int i) { return ld_cluster4(map_to_rank(po + r * D + c, i)); });
                finish<E, D, LIST>(p, u, u.rb * R + r, c, s);
            }
            __syncwarp();
            cluster_sync();                // parts stay until everyone has read them
            return;
        }
        const bool whole = count == sp.steps;
        const int slot = at == begin ? 0 : 1;
        const int live_rows = min(ROWS::kRows, p.rows - u.rb * ROWS::kRows);
        for (int i = tid; i < live_rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4));
            const Sums s = sum_parts<L::kTeams>(
                L::kTeams, [&](int t) { return sml[t * ROWS::kRows + r]; },
                [&](int t) { return *reinterpret_cast<const float4 *>(so + (t * ROWS::kRows + r) * D + c); });
            if (whole) {
                finish<E, D, LIST>(p, u, u.rb * ROWS::kRows + r, c, s);
            } else {
                const size_t pr = ((size_t)cta * 2 + slot) * ROWS::kRows + r;
                *reinterpret_cast<float4 *>(p.part_o + pr * D + c) = s.o;
                if (c == 0) p.part_ml[pr] = make_float2(s.m, s.l);
            }
        }
        if (step == 0 && tid == 0 && (p.by_unit || !whole)) {
            JoinRecord r;
            r.n = n;
            r.sub = sub;
            r.parts = whole ? 0 : cta_of(W, G, at + sp.steps - 1) - cta + 1;
            r.place = 2 * cta + slot;
            p.rec[p.by_unit ? n * p.units_per_seq + sub : cta] = r;
        }
        at += count;
        step = 0;
        if (at < end && ++sub == p.units_per_seq) {
            sub = 0;
            sp = span_of<LIST>(p, ++n);
        }
        __syncthreads();                   // the next unit loads into the ring
    }
}

template <typename E> __device__ __forceinline__ void store2(void *p, size_t i, float a, float b);
template <> __device__ __forceinline__ void store2<float>(void *p, size_t i, float a, float b) {
    *reinterpret_cast<float2 *>(static_cast<float *>(p) + i) = make_float2(a, b);
}
template <> __device__ __forceinline__ void store2<__nv_bfloat16>(void *p, size_t i, float a, float b) {
    *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p) + i) = pack2(a, b);
}

// Joins the parts of the units that more than one CTA ran, a record per blockIdx.x.  With few units
// (many parts each) a CTA takes row blockIdx.y, its warps taking the parts in turn; with many (one or
// two parts each) a warp takes a row, which keeps the grid small.
constexpr int kJoinWarps = 8;

template <typename E, int D, int ROWS, bool LIST, bool FEW>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_join_kernel(const __grid_constant__ DecodeParams p) {
    __shared__ float so[FEW ? kJoinWarps : 1][D];
    __shared__ float2 sml[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = FEW ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
    constexpr int V = D / 32, STEP = FEW ? kJoinWarps : 1;
    pdl_wait();
    const JoinRecord rec = p.rec[blockIdx.x];
    if (rec.parts < 2) return;
    const Unit u = unit_of<LIST>(p, rec.n, rec.sub);
    const int row = u.rb * ROWS + r;
    if (r >= ROWS || row >= p.rows) return;
    // this warp's parts: first, first + STEP, ..; a lane weighs one, and their outputs, which do not
    // wait for the weights, come in several at a time
    const int first = FEW ? warp : 0, count = rec.parts > first ? (rec.parts - first + STEP - 1) / STEP : 0;
    auto place = [&](int k) -> size_t {
        const int i = first + k * STEP;
        return (size_t)(i == 0 ? rec.place : (rec.place | 1) - 1 + 2 * i) * ROWS + r;
    };
    float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
    for (int k0 = 0; k0 < count; k0 += 32) {
        const float2 ml = k0 + lane < count ? p.part_ml[place(k0 + lane)] : make_float2(-INFINITY, 0.f);
        float mx = fmaxf(m, ml.x);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float shift = mx == -INFINITY ? 0.f : mx, old = ex2(m - shift), f = ex2(ml.x - shift);
        m = mx;
        l = l * old + warp_sum(ml.y * f);
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= old;
        const int n = min(32, count - k0);
#pragma unroll 8
        for (int k = 0; k < n; ++k) {
            const float g = __shfl_sync(0xffffffffu, f, k);
            const float *src = p.part_o + place(k0 + k) * D + lane * V;
            if constexpr (V == 4) {
                const float4 x = *reinterpret_cast<const float4 *>(src);
                o[0] = fmaf(x.x, g, o[0]);
                o[1] = fmaf(x.y, g, o[1]);
                o[2] = fmaf(x.z, g, o[2]);
                o[3] = fmaf(x.w, g, o[3]);
            } else {
                const float2 x = *reinterpret_cast<const float2 *>(src);
                o[0] = fmaf(x.x, g, o[0]);
                o[1] = fmaf(x.y, g, o[1]);
            }
        }
    }
    const size_t rh = row_head<LIST>(p, u, row);
    if (!FEW) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < V; e += 2) store2<E>(p.out, rh * D + lane * V + e, o[e] * inv, o[e + 1] * inv);
        if (lane == 0 && p.lse) p.lse[rh] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
        return;
    }
    if (lane == 0) sml[warp] = make_float2(m, l);
#pragma unroll
    for (int e = 0; e < V; ++e) so[FEW ? warp : 0][lane * V + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sml[w].x);
    const float shift = m == -INFINITY ? 0.f : m;
    const int col = 2 * threadIdx.x;
    float a = 0.f, b = 0.f;
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(sml[w].x - shift);
        l = fmaf(sml[w].y, f, l);
        a = fmaf(so[FEW ? w : 0][col], f, a);
        b = fmaf(so[FEW ? w : 0][col + 1], f, b);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    store2<E>(p.out, rh * D + col, a * inv, b * inv);
    if (threadIdx.x == 0 && p.lse) p.lse[rh] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

template <class ROWS, int D, bool LIST> PerDevice g_setup;
// clusters of 2 << i CTAs that run at once on a device
template <class ROWS, int D, bool LIST> int g_clusters[PerDevice::kMaxDevices][4];

template <class ROWS, int D, bool LIST>
cudaLaunchConfig_t cluster_config(cudaLaunchAttribute *cluster, long long units, int size,
                                  cudaStream_t stream) {
    cluster->id = cudaLaunchAttributeClusterDimension;
    cluster->val.clusterDim.x = size;
    cluster->val.clusterDim.y = cluster->val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<ROWS, D>::kSmem;
    cfg.stream = stream;
    cfg.attrs = cluster;
    cfg.numAttrs = 1;
    return cfg;
}

template <class ROWS, int D, bool LIST> cudaError_t setup() {
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    const auto line = attn_decode_kernel<ROWS, D, LIST, false>, in_cluster = attn_decode_kernel<ROWS, D, LIST, true>;
    constexpr int smem = Layout<ROWS, D>::kSmem;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(line, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(in_cluster, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(in_cluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
        cudaLaunchAttribute attr;
        const cudaLaunchConfig_t cfg = cluster_config<ROWS, D, LIST>(&attr, 1, 2 << i, nullptr);
        int &most = g_clusters<ROWS, D, LIST>[dev][i];
        if (cudaOccupancyMaxActiveClusters(&most, in_cluster, &cfg) != cudaSuccess) {
            most = 0;                      // a size the device does not take
            cudaGetLastError();
        }
    }
    return e;
}

// Most steps that a unit of the call can have.
template <bool LIST> long long most_steps(const DecodeParams &p) {
    if (LIST) return (p.list_len + kStep - 1) / kStep + (p.recent + kStep - 1) / kStep;
    long long tokens = (long long)p.cache.max_pages << p.cache.page_shift;
    if (p.window > 0 && tokens > (long long)p.window + p.T + kStep) tokens = (long long)p.window + p.T + kStep;
    return (tokens + kStep - 1) / kStep;
}

// CTAs of a cluster for each unit, or 1: the even split and its join. A cluster saves the second grid
// and the parts' way through memory, about 3 us or 5 steps, but gives every unit the same CTAs whatever
// its length, and some SMs none. (bf16, 16 x 2 heads, even split / cluster: 4 sequences of 1024 tokens 9.5 /
// 6.6 us; lists of 2048 for 8 sequences 11.1 / 10.1, for 16 14.5 / 11.1, for 32 20.2 / 16.0, for 74 36.8 /
// 33.2; but for 37 19.8 / 22.4, and 1 sequence of 16,384 tokens 13.4 / 15.9.)
// The table's width stands for the lengths: 4 sequences of 1024 tokens behind a table of 8192 take 7.2 us, and
// behind wider ones, where a sequence could be long, the even split's 9.4.
template <class ROWS, int D, bool LIST> int cluster_for(const DecodeParams &p, long long units, int grid) {
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    const long long steps = most_steps<LIST>(p);
    // (16 CTAs are worth their wider barrier for long units or few: 8 units of 16 steps 7.1 us, with 8 6.6)
    int i = steps > 32 || units <= 4 ? 3 : 2;
    while (i >= 0 && units > g_clusters<ROWS, D, LIST>[dev][i]) --i;
    if (i < 0) return 1;
    const int size = 2 << i;
    const long long each = (steps + size - 1) / size;
    // whole cache: the lengths behind the table's are not known, so a long sequence may be alone
    return each - units * steps / grid <= 5 && (LIST || each <= 8) ? size : 1;
}

template <class ROWS, int D, bool LIST>
cudaError_t launch_rows(DecodeParams p, void *workspace, cudaStream_t stream) {
    constexpr int smem = Layout<ROWS, D>::kSmem;
    int sms = 0;
    cudaError_t e = g_setup<ROWS, D, LIST>.ensure(setup<ROWS, D, LIST>, &sms);
    if (e != cudaSuccess) return e;
    // (fp32 rings of d = 128 leave room for one CTA an SM)
    const int grid = sms * (2 * (smem + 1024) <= 233472 ? kCtasPerSm : 1);
    p.row_blocks = (p.rows + ROWS::kRows - 1) / ROWS::kRows;
    p.units_per_seq = p.cache.H_kv * p.row_blocks * (LIST ? p.T : 1);
    const long long units = (long long)p.N * p.units_per_seq;
    const int size = cluster_for<ROWS, D, LIST>(p, units, grid);
    if (size > 1) {
        cudaLaunchAttribute attr;
        const cudaLaunchConfig_t cfg = cluster_config<ROWS, D, LIST>(&attr, units, size, stream);
        return cudaLaunchKernelEx(&cfg, attn_decode_kernel<ROWS, D, LIST, true>, p);
    }
    p.by_unit = units <= grid;
    p.rec = reinterpret_cast<JoinRecord *>(static_cast<unsigned char *>(workspace) + kErrorBytes);
    p.part_ml = reinterpret_cast<float2 *>(p.rec + grid);
    p.part_o = reinterpret_cast<float *>(p.part_ml + (size_t)grid * 2 * ROWS::kRows);
    attn_decode_kernel<ROWS, D, LIST, false><<<grid, kThreads, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int rows = p.rows < ROWS::kRows ? p.rows : ROWS::kRows;
    // (row to a CTA / to a warp: 1 sequence of 16,384 tokens x 2 heads 13.3 / 28.3 us a call, 4 of 32,768 x 4
    // 49.8 / 52.4, lists for 40 x 2 heads 22.4 / 23.9; lists for 100 x 2 50.7 / 49.5, 64 x 8 heads of 2048 tokens,
    // four drafts, 103 / 94)
    const bool few = units * 3 <= grid;
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.by_unit ? (unsigned)units : grid, few ? rows : (rows + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, attn_join_kernel<typename ROWS::E, D, ROWS::kRows, LIST, true>, p)
               : cudaLaunchKernelEx(&cfg, attn_join_kernel<typename ROWS::E, D, ROWS::kRows, LIST, false>, p);
}

template <int D, bool LIST>
cudaError_t launch_dim(const DecodeParams &p, bool bf16, void *ws, cudaStream_t stream) {
    if (bf16) {
        if (p.rows <= 16) return launch_rows<TensorRows<D, 1, LIST>, D, LIST>(p, ws, stream);
        if (p.rows <= 32) return launch_rows<TensorRows<D, 2, LIST>, D, LIST>(p, ws, stream);
        return launch_rows<TensorRows<D, 4, LIST>, D, LIST>(p, ws, stream);
    }
    if (p.rows == 1) return launch_rows<FmaRows<D, 1, LIST>, D, LIST>(p, ws, stream);
    if (p.rows <= 4) return launch_rows<FmaRows<D, 4, LIST>, D, LIST>(p, ws, stream);
    return launch_rows<FmaRows<D, 8, LIST>, D, LIST>(p, ws, stream);
}

constexpr int kMostRows = 64;              // largest ROWS::kRows

// Query rows that share a block of the prompt kernel (attn_prefill.cu): drafted tokens x packed heads.
int block_rows(int T, int G) {
    int pack = 1;
    while (pack < 16 && G % (2 * pack) == 0) pack *= 2;
    return T * pack;
}

// Whether a call's drafted tokens make enough rows for the prompt kernel, whose tcgen05 products take 128
// rows at the pace of one.  With more than 32 rows to a block of it, mma.sync row tiles no longer keep up
// with the cache; with fewer than 8 units the even split over all SMs wins all the same (1 sequence x 2
// heads x 8000 tokens, 64 rows: 19 against 24 us).
// That kernel gives every block the same CTAs, so the longest sequence sets its time, 12 us for each 1000
// tokens of a CTA, and lengths are not known here: only calls that cannot leave a CTA more than 64
// tokens to a row of its block take it, which keeps the loss on a skewed batch at the gain on an even one.
// (64 sequences x 2 heads, prompt kernel / even split.  At the limit: 64 rows, all of 4096 tokens 59 / 85 us,
// one among 512s 56 / 29; 128 rows, all of 8192 tokens 108 / 270, one among 1000s 106 / 57.  Past it: one of
// 262,144 among 1000s, 64 rows 3130 / 126, 128 rows 3140 / 208; 1000 to 32,768 tokens 391 / 290 and 399 / 540.)
bool many_rows(const gdn_paged_kv &kv, int N, int T, int H_q, int window, int sms) {
    const int rows = block_rows(T, H_q / kv.H_kv);
    if (rows <= 32 || (long long)N * kv.H_kv < 8) return false;
    long long tokens = (long long)kv.max_pages * kv.page_size;
    if (window > 0 && tokens > (long long)window + T) tokens = (long long)window + T;
    return tokens <= 64LL * rows * attn_prefill_splits(kv, N, (long long)N * T, H_q, sms);
}

}  // namespace

cudaError_t launch_attn_prefill(const gdn_paged_kv &kv, const void *q, const int32_t *cu,
                                const int32_t *pos0, const int32_t *prefix, void *out, float *lse,
                                int N, long long T_total, int H_q, float scale, float cap, int window,
                                void *workspace, size_t workspace_bytes, int sms, uint32_t budget,
                                cudaStream_t stream);

// `rows`: query rows that share a key head (H_q / H_kv x n_queries), blocked as launch_dim does.  Records
// and parts come behind the error word, which the prompt kernel and gdn_get_device_error take to be at the
// start of any workspace: a share more than the SMs' makes room for it.
size_t attn_decode_workspace_bytes(int rows, int d, int sms) {
    const size_t block = rows <= 16 ? 16 : rows <= 32 ? 32 : kMostRows;
    const size_t share = kCtasPerSm * (sizeof(JoinRecord) + 2 * block * (sizeof(float2) + d * sizeof(float)));
    static_assert(kErrorBytes <= kCtasPerSm * 2 * 16 * sizeof(float2), "the error word fits the least share");
    const size_t own = (size_t)(sms + 1) * share;
    // (a call that the prompt kernel takes needs a little more for its table of blocks)
    return rows > 32 ? own + ((size_t)64 << 10) : own;
}

cudaError_t launch_attn_decode(const gdn_paged_kv &kv, const void *q, const int32_t *q_pos,
                               const int32_t *list, int list_len, int recent, bool lists,
                               void *out, float *lse, int N, int T, int H_q, float scale,
                               float cap, int window, void *workspace, size_t workspace_bytes,
                               int sms, uint32_t budget, cudaStream_t stream) {
    if (!lists && kv.dtype == GDN_BF16 && many_rows(kv, N, T, H_q, window, sms))
        return launch_attn_prefill(kv, q, nullptr, q_pos, nullptr, out, lse, N, (long long)N * T, H_q,
                                   scale, cap, window, workspace, workspace_bytes, sms, budget, stream);
    DecodeParams p = {};
    p.cache = paged_view(kv);
    p.q = q;
    p.q_pos = q_pos;
    p.list = list;
    p.out = out;
    p.lse = lse;
    p.N = N;
    p.T = T;
    p.H_q = H_q;
    p.G = H_q / kv.H_kv;
    p.rows = lists ? p.G : p.G * T;
    p.list_len = list_len;
    p.recent = recent;
    p.window = window;
    p.score = scoring(scale, cap);
    const bool bf16 = kv.dtype == GDN_BF16;
    if (kv.d == 128)
        return lists ? launch_dim<128, true>(p, bf16, workspace, stream)
                     : launch_dim<128, false>(p, bf16, workspace, stream);
    return lists ? launch_dim<64, true>(p, bf16, workspace, stream)
                 : launch_dim<64, false>(p, bf16, workspace, stream);
}

}  // namespace gdn
