// gdn_attn_prefill (include/attn.h), bf16: attention of prompts over the paged cache on the
// tcgen05 tensor cores.
//
//   S = Q K^T,  x = cap(scale S),  m = running row maximum,  P = e^{x - m},
//   O <- O e^{m_old - m} + P V,  l <- l e^{m_old - m} + sum P,   out = O / l
//
// A CTA owns 256 query rows that share one key head: the tokens of a block, each with `pack`
// heads (a power of two that divides the group), so a K / V tile in shared memory serves all of
// them and the causal edge of the block is 256 / pack tokens wide.  Rows form two tiles of 128
// whose products and exponentials alternate:
//
//   tensor:   S_A(j+1)  PV_B(j)  S_B(j+1)  PV_A(j+1)  ...
//   warps:    softmax B(j)       softmax A(j+1)       ...
//
// Per pair of 128 x 128 tiles (d = 128) the tensor pipe needs 2048 cycles and the 2 x 16384
// exponentials, at 16 per cycle and SM, 2048 as well: the two are balanced, and what is lost is
// what does not overlap. A pair takes about 3100 cycles: of a tile's turn (loads of S, maxima, 1024
// cycles of exponentials, then PV and the next S) only the other tile's products lie beside it, since
// two S, two O fill TMEM and S(j+1) cannot start before PV(j) has read P(j). (A quarter of the
// exponentials as polynomials on the FMA pipe made it longer, 126 -> 133 us at 2 x 4096 tokens.)
//  - warps 0-3, 4-7: the softmax of tile A, B; a thread owns a row (TMEM lane), so maxima and
//    sums need no exchange.  P goes back to TMEM over the first half of S, as the A operand of PV.
//    O is rescaled only when a row's maximum grew by more than 2^8 (until then P and l simply use
//    the old one): after the first tiles that is rare, so no warps are kept for it.
//  - warp 8: issues the products.  PV(j) and S(j+1) of a tile go out together; S(j+1) overwrites the
//    columns P(j) was in, after PV(j) read them (one thread's products run in order).
//  - warp 10: loads.  K and V tiles of 128 tokens alternate through a ring of four, gathered page by
//    page with TMA; tokens that are absent are left out of the softmax by a mask, and their V rows (and
//    those past the sequence) are zeroed, so nothing a dead row holds reaches a product.
//  - warps 9 and 11 fill the warpgroup, whose registers the softmax takes over.
//
// Measured: one prompt of 16,384 tokens x 16 heads (2 key heads) 855-910 us, 1.21-1.29 PFLOP/s on a
// chip at its power cap (cuBLAS there: 1.40); 2 x 4096 tokens 126 us, 1.09 PFLOP/s, tensor pipe active
// 49%; d = 64: 16,384 tokens 726 us, 0.76 PFLOP/s, 2 x 4096 111 us, 0.62, with as many exponentials
// (that pipe active 61%) for half the products; a window of 1024 over 16,384 tokens 176 us, 0.76 PFLOP/s;
// 8191 ragged tokens behind 2800-4000, 16 x 4 heads, capped, pages of 16: 398 us. Of these the cap
// takes 60 (the FMA pipe), pages of 16 rather than 128 tokens 30 (eight loads to a tile half), and
// unequal blocks on 148 SMs 40.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "attn_prefill.cuh"
#include "device_once.h"
#include "sm100.cuh"

namespace gdn {
using namespace sm100;

namespace {

constexpr int kThreads = 384, kSlots = 4, kMaskRing = 8;
// Registers a thread: 168 at launch (384 threads); the softmax warps, which hold a row of scores,
// take what the third warpgroup gives up: 2 x 208 + 88 = 3 x 168.
constexpr int kRegsSoftmax = 208, kRegsOther = 88;
constexpr int kTile = kPrefillTile;        // query rows of a tile, tokens of a K / V tile
constexpr uint32_t kPollNs = 2000, kDrainBudget = GDN_DEFAULT_WAIT_BUDGET;
constexpr float kLazy = 8.f;               // growth of a row maximum (base 2) that O may lag

// cap2 tanh(k s) + add for two s, by the polynomial of degree DEG whose coefficients carry k and cap2
template <int DEG> struct Near {
    float c[DEG + 1];
    __device__ __forceinline__ Near(float k, float cap2) {
        float f = k * cap2;
#pragma unroll
        for (int i = 0; i <= DEG; ++i, f *= k * k) c[i] = tanh_r<DEG>(i) * f;
    }
    __device__ __forceinline__ float2 operator()(float2 s, float2 add) const {
        const float2 t = mul2(s, s);
        float2 r = make_float2(c[DEG], c[DEG]);
#pragma unroll
        for (int i = DEG - 1; i >= 0; --i) r = fma2(r, t, make_float2(c[i], c[i]));
        return fma2(s, r, add);
    }
};
// the larger of three
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

enum Bar {
    B_Q = 0, B_FULL = 1, B_EMPTY = B_FULL + kSlots, B_S = B_EMPTY + kSlots, B_P = B_S + 2,
    B_O = B_P + 4, B_FIX = B_O + 2, B_DRAIN, B_COUNT                    // B_P: tile x part
};

template <int D>
struct Smem {
    static constexpr uint32_t kHalf = kTile * 128;             // 64 dims of a tile
    static constexpr uint32_t kTileBytes = (D / 64) * kHalf;
    static constexpr uint32_t kQ = 0, kRing = 2 * kTileBytes;
    static constexpr uint32_t kMask = kRing + kSlots * kTileBytes;
    static constexpr uint32_t kBars = kMask + kMaskRing * 16;
    static constexpr uint32_t kMisc = kBars + 8 * ((B_COUNT + 1) / 2 * 2);
    static constexpr uint32_t kTotal = kMisc + 16 + 1024;       // 1024: alignment of the base
};
constexpr uint32_t kTmS = 0, kTmO = 256;                        // TMEM columns, 128 per tile each

template <int N> __device__ __forceinline__ void regs_take() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_give() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, uint32_t budget,
                                          const volatile int *abort_flag) {
    for (uint32_t i = 0; i < budget; ++i) {
        // (the timed form costs a few hundred cycles even when the phase is over)
        if (i < 64 ? mbar_try_wait(bar, parity) : mbar_try_wait_sleep(bar, parity, kPollNs)) return true;
        if (*abort_flag) return false;
    }
    return false;
}

// What the outputs need of a block, kept in shared memory while the registers hold scores.
struct Outputs {
    long long first;                       // row of the sequence's first token
    int len, q0, h0;                       // its tokens; the block's first token and query head
    int parts, part;                       // CTAs that share the block; this one's place among all parts
};

template <int D, bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v,
                    const __grid_constant__ AttnPrefillParams p) {
    using L = Smem<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ Outputs block_outputs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bt_tile = kTile >> p.pack_shift, bt = 2 * bt_tile;        // tokens of a tile, block
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kBars);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::kMisc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::kMisc + 4);
    // set up while the block's sequence is being found
    if (warp == 8) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
    if (tid < 32 * 10 && tid >= 32 * 9) {
        if (lane == 0) { prefetch_map(&tm_q); prefetch_map(&tm_k); prefetch_map(&tm_v); }
        for (int b = lane; b < B_COUNT; b += 32) mbar_init(bars + b, b >= B_P && b < B_P + 4 ? 4 : 1);
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    pdl_trigger();
    int n, blk;
    Sequence seq;
    const int packs = p.G >> p.pack_shift, heads = p.cache.H_kv * packs;
    // Heads take turns when one head's blocks do not fill the SMs (so the longest blocks of all of
    // them start first: 442 against 474 us on 137 blocks x 4 heads), and follow one another when
    // they do (then all SMs read the same K and V: 126 against 130 us on 256 blocks x 2 heads).
    const int block = blockIdx.x / p.splits, split = blockIdx.x % p.splits, blocks = gridDim.x / p.splits / heads;
    const int hx = p.heads_first ? block % heads : block / blocks;
    const bool found = find_block<kThreads>(p, [&](long long len) { return (len + bt - 1) / bt; },
                                            p.heads_first ? block / heads : block % blocks, n, blk, seq);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!found) {
        if (p.splits > 1 && split == 0 && tid == 0) p.split_blocks[block].parts = 0;
        if (warp == 8) tmem_dealloc(tmem, 512);
        return;
    }
    const int hk = hx / packs;                                           // key head
    const int h0 = hk * p.G + (hx % packs << p.pack_shift);              // first query head
    const long long first = seq.first;
    const int len = seq.len;
    const Sight see(p, seq);
    const int e = see.e;
    const int q0 = blk * bt;
    const int k_lo = see.lo(q0);                                         // oldest token seen
    int k_base = k_lo / kTile * kTile;
    auto tiles_of = [&](int i) -> int {                                  // K / V tiles row tile i walks
        const int a = q0 + i * bt_tile;
        const int hi = a < len ? see.hi(min(a + bt_tile, len) - 1) : 0;
        return hi > k_base ? (hi - k_base - 1) / kTile + 1 : 0;
    };
    int tiles_a = tiles_of(0), tiles_b = tiles_of(1), nt = max(tiles_a, tiles_b);
    int parts = 1;
    if (p.splits > 1) {
        parts = split_parts(nt, p.splits);
        if (split == 0 && tid == 0)
            p.split_blocks[block] = SplitBlock{first, len, q0 << p.pack_shift, 1 << p.pack_shift, h0, parts, 0};
        if (split >= parts) {
            if (warp == 8) tmem_dealloc(tmem, 512);
            return;
        }
        int from, to;
        split_range(nt, parts, split, from, to);
        k_base += from * kTile;
        nt = to - from;
        tiles_a = min(max(tiles_a - from, 0), nt);
        tiles_b = min(max(tiles_b - from, 0), nt);
    }

    if (tid == 0) block_outputs = Outputs{first, len, q0, h0, parts, block * p.splits + split};
    __syncthreads();
    auto wait = [&](int b, int k) -> bool {                              // k-th completion of barrier b
        return wait_bounded(bars + b, (uint32_t)(k & 1), p.budget, abort_flag);
    };
    auto fail = [&](int where) {
        if (!*abort_flag) {
            *abort_flag = 1;
            record_error(p.err, GDN_ERR_TIMEOUT, where);
        }
    };

    if (warp < 8) {
        // ==================================================================== softmax
        regs_take<kRegsSoftmax>();
        const int i = warp >> 2, row = tid & 127, tiles = i ? tiles_b : tiles_a;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t s_at = tmem + lanes + kTmS + 128 * i, o_at = tmem + lanes + kTmO + 128 * i;
        const int tok = q0 + i * bt_tile + (row >> p.pack_shift);
        const int lo = see.lo(tok), hi = see.hi(tok);
        // tiles that every row of this row tile sees whole
        const int lo_max = see.lo(q0 + (i + 1) * bt_tile - 1), hi_min = see.hi(q0 + i * bt_tile);
        float m = -INFINITY, l = 0.f;                                    // m in base-2 units
        bool ok = true;
        // |mul|: the products carry the scale's sign.  A scale of 0 makes every score equal, and so
        // does 1e-30, which keeps -inf (a masked score) times it -inf.
        const float k2 = CAP ? fabsf(p.score.mul) : fmaxf(fabsf(p.score.mul), 1e-30f);
        const float cap2 = p.score.cap2;
#pragma unroll 1
        for (int j = 0; j < tiles; ++j) {
            if (!__all_sync(0xffffffffu, wait(B_S + i, j))) { fail(1 + i); ok = false; break; }
            tc_fence_after();
            uint32_t raw[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, raw[c]);
            const int k0 = k_base + j * kTile;
            const uint4 pm = *reinterpret_cast<const uint4 *>(sm + L::kMask + (j % kMaskRing) * 16);
            tmem_wait_ld();
            float s[128];
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(raw[c >> 5][c & 31]);
            const bool whole = k0 >= lo_max && k0 <= hi_min - kTile &&
                               (pm.x & pm.y & pm.z & pm.w) == 0xffffffffu;
            uint32_t live[4] = {pm.x, pm.y, pm.z, pm.w};
            if (!whole) {
                const int a = lo - k0, z = hi - k0;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    // bits of tokens [a, z) of this word
                    const int b0 = min(max(a - 32 * w, 0), 32), b1 = min(max(z - 32 * w, 0), 32);
                    const uint32_t below1 = b1 == 32 ? 0xffffffffu : (1u << b1) - 1u;
                    const uint32_t below0 = b0 == 32 ? 0xffffffffu : (1u << b0) - 1u;
                    live[w] &= below1 & ~below0;
                }
            }
            // tanh(y) by a polynomial on the FMA pipe while no live score of the warp's rows passes the
            // cap (|y| <= 1), a shorter one while none passes half of it, else by exponentials too (two
            // more per score on the busiest pipe: 383 against 185 us for 2 x 1500 tokens behind 4000, 16 x
            // 4 heads; 155 without a cap). In whole tiles the polynomial runs beside the weights'
            // exponentials, with the scale in its coefficients (8191 tokens behind 2800-4000, 16 x 4 heads:
            // 404 us, 412 with a product more per score).
            bool near = false, nearer = false;
            if (CAP) {
                float far = 0.f;
                if (whole) {
#pragma unroll
                    for (int c = 0; c < 128; c += 2) far = max3(far, fabsf(s[c]), fabsf(s[c + 1]));
                } else {
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        far = fmaxf(far, (live[c >> 5] >> (c & 31)) & 1 ? fabsf(s[c]) : 0.f);
                }
                near = __all_sync(0xffffffffu, far * k2 <= p.near_at);
                nearer = whole && __all_sync(0xffffffffu, far * k2 <= p.nearer_at);
                // in place, two at a time
                auto cap_all = [&](auto &&cap) {
#pragma unroll
                    for (int c = 0; c < 128; c += 2) {
                        const float2 x = cap(mul2(make_float2(s[c], s[c + 1]), make_float2(k2, k2)));
                        s[c] = x.x;
                        s[c + 1] = x.y;
                    }
                };
                if (!near) cap_all([&](float2 y) { return capped2<3>(y, cap2); });
                else if (!whole) cap_all([&](float2 y) { return capped_near2<5>(y, cap2); });
                near = near && whole;
            }
            if (!whole) {
#pragma unroll
                for (int c = 0; c < 128; ++c) s[c] = (live[c >> 5] >> (c & 31)) & 1 ? s[c] : -INFINITY;
            }
            float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 124; c += 8)
#pragma unroll
                for (int x = 0; x < 4; ++x) mx4[x] = max3(mx4[x], s[c + x], s[c + 4 + x]);
            float mx = max3(fmaxf(mx4[0], s[124]), fmaxf(mx4[1], s[125]),
                            fmaxf(fmaxf(mx4[2], s[126]), fmaxf(mx4[3], s[127])));
            if (CAP ? near : mx != -INFINITY) mx = CAP ? capped_near2<5>(make_float2(mx * k2, 0.f), cap2).x : mx * k2;
            const bool grow = mx > m + kLazy;                            // also when m is -inf
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2(m - mx) : 1.f;                // 0 from -inf
                if (grow) m = mx;
                l *= f;
                if (j > 0) {
                    // PV(j - 1) is complete: S(j) was issued after it and has arrived
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(o_at + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                        tmem_st32(o_at + 32 * c, o);
                    }
                }
            }
            const float shift = m == -INFINITY ? 0.f : m;
            // Each weight is rounded to bf16 for the product (off by 2^-8 of itself at most); the
            // sum takes the unrounded ones.  P goes out in two parts: PV of the first 96 tokens
            // runs while the last 32 weights are formed.
            const float2 kk = make_float2(CAP ? 1.f : k2, CAP ? 1.f : k2), sh = make_float2(-shift, -shift);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto publish = [&](int part) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_local(bars + B_P + 2 * i + part);
            };
            auto all_weights = [&](auto &&exponent) {
                auto weights = [&](int at) -> uint32_t {
                    const float2 x = exponent(make_float2(s[at], s[at + 1]));
                    const float2 w = make_float2(ex2(x.x), ex2(x.y));
                    sum[at >> 1 & 1] = add2(sum[at >> 1 & 1], w);
                    return pack2(w.x, w.y);
                };
                uint32_t w32[32], w16[16];
#pragma unroll
                for (int x = 0; x < 32; ++x) w32[x] = weights(2 * x);
                tmem_st32(s_at, w32);
#pragma unroll
                for (int x = 0; x < 16; ++x) w16[x] = weights(64 + 2 * x);
                tmem_st16(s_at + 32, w16);
                publish(0);
#pragma unroll
                for (int x = 0; x < 16; ++x) w16[x] = weights(96 + 2 * x);
                tmem_st16(s_at + 48, w16);
            };
            if (CAP && nearer) {
                const Near<3> cap(k2, cap2);
                all_weights([&](float2 x) { return cap(x, sh); });
            } else if (CAP && near && p.nearer_at > 0.f) {
                const Near<5> cap(k2, cap2);
                all_weights([&](float2 x) { return cap(x, sh); });
            } else if (CAP && near) {
                const Near<2> cap(k2, cap2);
                all_weights([&](float2 x) { return cap(x, sh); });
            } else
                all_weights([&](float2 x) { return fma2(x, kk, sh); });
            l += sum[0].x + sum[0].y + sum[1].x + sum[1].y;
            publish(1);
        }
        if (ok && tiles > 0 && !__all_sync(0xffffffffu, wait(B_O + i, 0))) {
            fail(3 + i);
            ok = false;
        }
        if (ok) {
            tc_fence_after();
            const volatile Outputs &to = block_outputs;
            const long long first_row = to.first;
            const int tokens = to.len, token0 = to.q0 + i * bt_tile, head0 = to.h0, pack_mask = (1 << p.pack_shift) - 1;
            if (to.parts > 1) {
                // this CTA's share: unnormalised, in fp32 (a thread writes 128 bytes at a time)
                const size_t at = (size_t)to.part * 2 * kTile + i * kTile + row;
                p.part_ml[at] = make_float2(m, l);
#pragma unroll 1
                for (int c = 0; c < (tiles > 0 ? D / 32 : 0); ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_at + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<uint4 *>(p.part_o + at * D + 32 * c + 4 * x) =
                            make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                }
            } else {
                // A thread's row goes through the tile's Q, which nobody reads any more (in the same
                // swizzle), so that the warp stores whole rows.
                const float inv = l > 0.f ? 1.f / l : 0.f;
                unsigned char *stage = sm + L::kQ + i * L::kTileBytes;
#pragma unroll 1
                for (int c = 0; c < (tiles > 0 ? D / 32 : 0); ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_at + 32 * c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        uint32_t w[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            w[y] = pack2(__uint_as_float(o[8 * x + 2 * y]) * inv,
                                         __uint_as_float(o[8 * x + 2 * y + 1]) * inv);
                        *reinterpret_cast<uint4 *>(stage + (c >> 1) * L::kHalf + sw128(row, 4 * (c & 1) + x)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncwarp();
                constexpr int CH = D / 8, RPI = 32 / CH;                 // chunks of a row, rows at a time
                const int ch = lane % CH;
#pragma unroll 4
                for (int r0 = 0; r0 < 32; r0 += RPI) {
                    const int r = 32 * (warp & 3) + r0 + lane / CH;
                    const int t = token0 + (r >> p.pack_shift), h = head0 + (r & pack_mask);
                    const uint4 x = tiles > 0 ? *reinterpret_cast<const uint4 *>(stage + (ch >> 3) * L::kHalf + sw128(r, ch & 7))
                                              : make_uint4(0, 0, 0, 0);
                    if (t < tokens)
                        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                                   ((size_t)(first_row + t) * p.H_q + h) * D + 8 * ch) = x;
                }
                const int t = token0 + (row >> p.pack_shift);
                if (p.lse && t < tokens)
                    p.lse[(size_t)(first_row + t) * p.H_q + head0 + (row & pack_mask)] =
                        l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            }
        }
    } else {
        regs_give<kRegsOther>();
        if (warp == 8) {
            // =============================================================== products
            // Tile A's and tile B's turns alternate, which keeps the two softmax warpgroups half a period
            // apart (one issuing warp for each lets them fall into step).  The whole warp walks this code
            // and one elected lane issues: descriptors then stay in uniform registers (issued from a
            // divergent thread, a product took 60-100 cycles).
            const uint32_t neg = p.score.mul < 0.f ? 1u << 14 : 0u;      // the softmax takes |mul|
            const uint32_t id_s = idesc_bf16(128, 128, false, false) | neg;
            const uint32_t id_o = idesc_bf16(128, D, false, true);
            const uint64_t q_desc = sdesc_kmajor(smem_u32(sm + L::kQ));
            const uint64_t k_desc = sdesc_kmajor(smem_u32(sm + L::kRing));
            const uint64_t v_desc = sdesc_mnmajor(smem_u32(sm + L::kRing), L::kHalf);
            const bool leader = elect_one();
            auto scores = [&](int i, int slot) {
                const uint64_t a = q_desc + i * (L::kTileBytes >> 4), b = k_desc + slot * (L::kTileBytes >> 4);
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks) {
                        const uint32_t off = ((ks >> 2) * L::kHalf + (ks & 3) * 32) >> 4;
                        umma_bf16(tmem + kTmS + 128 * i, a + off, b + off, id_s, ks > 0);
                    }
                }
            };
            auto commit = [&](int b) { if (leader) umma_commit(bars + b); };
            auto ready = [&](int b, int k) -> bool { return __all_sync(0xffffffffu, wait(b, k)); };
            bool ok = true;
            int issued = 0;
            if (nt > 0 && (ok = ready(B_Q, 0) && ready(B_FULL, 0))) {
                tc_fence_after();
                issued = 1;
                if (tiles_a > 0) { scores(0, 0); commit(B_S); }
                if (tiles_b > 0) { scores(1, 0); commit(B_S + 1); }
                commit(B_EMPTY);
            }
#pragma unroll 1
            for (int j = 0; ok && j < nt; ++j) {
                const int vs = (2 * j + 1) % kSlots, ks = (2 * j + 2) % kSlots;
                const uint64_t b = v_desc + vs * (L::kTileBytes >> 4);
                ok = ready(B_FULL + vs, (2 * j + 1) / kSlots);
                if (ok && j + 1 < nt) ok = ready(B_FULL + ks, (2 * j + 2) / kSlots);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int tiles = i ? tiles_b : tiles_a;
                    const uint32_t s_at = tmem + kTmS + 128 * i, o_at = tmem + kTmO + 128 * i;
                    if (!ok || j >= tiles) continue;
                    if (!(ok = ready(B_P + 2 * i, j))) continue;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 6; ++k)
                            umma_bf16_ta(o_at, s_at + 8 * k, b + k * (2048 >> 4), id_o, j > 0 || k > 0);
                    }
                    if (!(ok = ready(B_P + 2 * i + 1, j))) continue;
                    tc_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 6; k < 8; ++k)
                            umma_bf16_ta(o_at, s_at + 8 * k, b + k * (2048 >> 4), id_o, 1);
                    }
                    if (j + 1 < tiles) scores(i, ks);
                    commit((j + 1 < tiles ? B_S : B_O) + i);
                }
                if (!ok) break;
                commit(B_EMPTY + vs);
                if (j + 1 < nt) commit(B_EMPTY + ks);
            }
            if (!ok) {
                if (lane == 0) fail(5);
                if (issued) {                                            // let the products end first
                    commit(B_DRAIN);
                    mbar_wait(bars + B_DRAIN, 0, kDrainBudget);
                }
            } else {
                // so they do here, also when the softmax warps give up on the last ones
                if (tiles_a > 0) mbar_wait(bars + B_O, 0, kDrainBudget);
                if (tiles_b > 0) mbar_wait(bars + B_O + 1, 0, kDrainBudget);
            }
            __syncwarp();
        } else if (warp == 10) {
        // ====================================================================== loads
        const int ps = 1 << p.cache.page_shift, box = ps < kTile ? ps : kTile;
        const int boxes = kTile / box;
        const bool leader = elect_one();
        if (nt > 0) {
            if (lane == 0) {
                mbar_arrive_expect_tx(bars + B_Q, 2 * L::kTileBytes);
                for (int i = 0; i < 2; ++i)
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_3d(sm + L::kQ + i * L::kTileBytes + h * L::kHalf, &tm_q, bars + B_Q,
                                    64 * h, h0, (int)(first + q0 + i * bt_tile));
            }
            bool ok = true;
            int done = 0, fixes = 0;                                     // slots handed on; V tiles patched
            bool patching = false;
#pragma unroll 1
            for (int j = 0; ok && j < nt; ++j) {
                const int k0 = k_base + j * kTile;
                const int t = k0 + min(lane, boxes - 1) * box;
                const int src = lane < boxes && t < e ? cache_row(p.cache, n, t) : -1;
                const uint32_t there = __ballot_sync(0xffffffffu, src >= 0);
                const uint32_t bytes = __popc(there) * box * D * 2;
                const bool patch = __popc(there) < boxes || k0 > e - kTile || k0 < k_lo;
                if (lane < 4) {
                    // presence, 32 tokens a word (a box is at least 16 tokens)
                    const uint32_t a = (there >> (32 * lane / box)) & 1, b = (there >> ((32 * lane + 16) / box)) & 1;
                    reinterpret_cast<uint32_t *>(sm + L::kMask + (j % kMaskRing) * 16)[lane] =
                        (a ? 0xffffu : 0u) | (b ? 0xffff0000u : 0u);
                }
                __syncwarp();                                            // before lane 0 arrives for K
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    const int use = 2 * j + v, slot = use % kSlots;
                    unsigned char *dst = sm + L::kRing + slot * L::kTileBytes;
                    if (use >= kSlots) ok = wait(B_EMPTY + slot, use / kSlots - 1);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    const bool fix = v && patch;
                    uint64_t *bar = bars + (fix ? B_FIX : B_FULL + slot);
                    if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    // the whole warp walks the boxes and one lane issues, as for the products (pages of 16
                    // tokens: 400 against 404 us with a lane to a box)
                    for (int b = 0; b < boxes; ++b) {
                        const int at = __shfl_sync(0xffffffffu, src, b);
                        if (at >= 0 && leader)
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_3d(dst + h * L::kHalf + b * box * 128, v ? &tm_v : &tm_k, bar,
                                            64 * h, hk, at);
                    }
                    if (fix) {
                        patching = true;
                        ok = wait(B_FIX, fixes);
                        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                        patching = false;
                        ++fixes;
                        for (int r = lane; r < kTile; r += 32)
                            if (k0 + r >= e || k0 + r < k_lo || !((there >> (r / box)) & 1))
                                for (int h = 0; h < D / 64; ++h)
#pragma unroll
                                    for (int c = 0; c < 8; ++c)
                                        *reinterpret_cast<uint4 *>(dst + h * L::kHalf + r * 128 + 16 * c) =
                                            make_uint4(0, 0, 0, 0);
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_local(bars + B_FULL + slot);
                    }
                    ++done;
                }
            }
            if (!ok) {
                if (lane == 0) fail(6);
                __syncwarp();
            }
            // This CTA's copies land before its shared memory is released, also when another warp gives
            // up on one after this point.
            mbar_wait(bars + B_Q, 0, kDrainBudget);
            if (patching) mbar_wait(bars + B_FIX, (uint32_t)(fixes & 1), kDrainBudget);
            for (int s = max(0, done - kSlots); s < done; ++s)
                mbar_wait(bars + B_FULL + s % kSlots, (uint32_t)(s / kSlots & 1), kDrainBudget);
        }
        __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult r;
        void *f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

// [rows, heads, d] bf16, boxes of 64 dims x box_heads x box_rows in the 128-byte swizzle
bool make_map(CUtensorMap *map, const void *base, long long rows, int heads, int d, int box_heads,
              int box_rows) {
    auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)heads * d * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t one[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool CAP> PerDevice g_setup;

template <int D, bool CAP>
cudaError_t launch_dim(AttnPrefillParams p, const gdn_paged_kv &kv, cudaStream_t stream) {
    constexpr int smem = Smem<D>::kTotal;
    int sms = 0;
    cudaError_t e = g_setup<D, CAP>.ensure([] {
        return cudaFuncSetAttribute(attn_prefill_kernel<D, CAP>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    }, &sms);
    if (e != cudaSuccess) return e;
    const int pack = 1 << p.pack_shift;
    const int box = kv.page_size < kTile ? kv.page_size : kTile;
    const long long rows = (long long)kv.num_pages * kv.page_size;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, p.q, p.T_total, p.H_q, D, pack, kTile / pack) ||
        !make_map(&mk, kv.k, rows, kv.H_kv, D, 1, box) ||
        !make_map(&mv, kv.v, rows, kv.H_kv, D, 1, box))
        return cudaErrorInvalidValue;
    p.heads_first = p.blocks / (kv.H_kv * (p.G >> p.pack_shift)) < sms;
    attn_prefill_kernel<D, CAP><<<(unsigned)(p.blocks * p.splits), kThreads, smem, stream>>>(mq, mk, mv, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_bf16(const AttnPrefillParams &p, const gdn_paged_kv &kv, cudaStream_t stream) {
    const bool cap = p.score.cap2 != 0.f;
    if (kv.d == 128) return cap ? launch_dim<128, true>(p, kv, stream) : launch_dim<128, false>(p, kv, stream);
    return cap ? launch_dim<64, true>(p, kv, stream) : launch_dim<64, false>(p, kv, stream);
}

}  // namespace gdn
