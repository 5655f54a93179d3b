// gdn_attn_prefill (include/attn.h), fp32: the same attention on the CUDA cores, since one product of
// operands of fewer bits would not hold fp32's tolerance (operands as sums of bf16 parts were not tried).
//
// A CTA owns 64 query rows of one key head (row r of a sequence: token r / G, head r % G of the
// group) and walks the tokens they see in tiles of 64, with a running maximum and sum.  Thread
// (ty, tx) of 16 x 16 holds the scores of rows 4 ty + a and keys tx + 16 b, and the outputs of the
// same rows and D / 16 dims, so a row's maxima and sums stay inside a half warp.  Both products run
// from shared memory, two FMAs to an instruction.  The weights take the place of the keys they came
// from, which lets two CTAs share an SM at d = 128, so that one's products cover the other's loads
// (2 x 2048 tokens, 8 x 2 heads: 466 us, 37 TFLOP/s; 571 with a place of their own and one CTA an SM,
// 606 with single FMAs besides; d = 64 265 us, 32 TFLOP/s; one of 8192 tokens with a window of 1024 953 us,
// 34).  A thread's 4 x 4 scores take eight 16-byte reads of shared memory to 32 packed FMAs, and those reads,
// not the FMA pipe, which runs at half its rate, set the pace.
#include <stdint.h>

#include "attn_prefill.cuh"
#include "device_once.h"

namespace gdn {
namespace {

constexpr int kThreads = 256, kRows = kF32Rows, kKeys = kF32Keys;

template <int D>
struct Smem {
    static constexpr int kPitch = D + 4;                     // rows of Q and K: no bank conflicts
    static constexpr int kQ = 0, kK = kQ + kRows * kPitch, kV = kK + kKeys * kPitch, kRow = kV + kKeys * D;
    static constexpr int kP = kK;                            // the weights follow the keys they came from
    static constexpr int kBytes = (kRow + kKeys) * 4;
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
attn_prefill_f32_kernel(const __grid_constant__ AttnPrefillParams p) {
    using L = Smem<D>;
    extern __shared__ float sm[];
    float *sq = sm + L::kQ, *sk = sm + L::kK, *sv = sm + L::kV, *sp = sm + L::kP;
    int *rows = reinterpret_cast<int *>(sm + L::kRow);       // cache row of each key, -1 absent
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    pdl_trigger();
    const int block = blockIdx.x / p.splits, split = blockIdx.x % p.splits;
    const int hk = block % p.cache.H_kv;
    int n, blk;
    Sequence seq;
    if (!find_block<kThreads>(p, [&](long long len) { return (len * p.G + kRows - 1) / kRows; },
                              block / p.cache.H_kv, n, blk, seq)) {
        if (p.splits > 1 && split == 0 && tid == 0) p.split_blocks[block].parts = 0;
        return;
    }
    const Sight see(p, seq);
    const long long r0 = (long long)blk * kRows, r_end = (long long)seq.len * p.G;
    const int t_first = (int)(r0 / p.G), t_last = (int)((min(r0 + kRows, r_end) - 1) / p.G);
    const int k_hi = see.hi(t_last);
    int k_lo = see.lo(t_first), parts = 1;
    int tiles = k_hi > k_lo ? (k_hi - k_lo - 1) / kKeys + 1 : 0;
    if (p.splits > 1) {
        parts = split_parts(tiles, p.splits);
        if (split == 0 && tid == 0)
            p.split_blocks[block] = SplitBlock{seq.first, seq.len, blk * kRows, p.G, hk * p.G, parts, 0};
        if (split >= parts) return;
        int from, to;
        split_range(tiles, parts, split, from, to);
        k_lo += from * kKeys;
        tiles = to - from;
    }
    auto row_at = [&](long long r) -> size_t {
        return (size_t)(seq.first + r / p.G) * p.H_q + (size_t)hk * p.G + r % p.G;
    };
    constexpr int C4 = D / 4;
    for (int i = tid; i < kRows * C4; i += kThreads) {
        const long long r = r0 + i / C4;
        const float4 x = r < r_end ? __ldg(reinterpret_cast<const float4 *>(p.q) + row_at(r) * C4 + i % C4)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4 *>(sq + (i / C4) * L::kPitch + 4 * (i % C4)) = x;
    }
    int lo[4], hi[4];
    float m[4], l[4];
    float2 o[4][D / 32];                                     // dims 64 d + 4 tx + (0, 1), (2, 3)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const long long r = r0 + 4 * ty + a;
        const int t = (int)(min(r, r_end - 1) / p.G);
        lo[a] = see.lo(t);
        hi[a] = see.hi(t);
        m[a] = -INFINITY;
        l[a] = 0.f;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[a][d] = make_float2(0.f, 0.f);
    }
    const float *kc = reinterpret_cast<const float *>(p.cache.k), *vc = reinterpret_cast<const float *>(p.cache.v);
    for (int i = 0; i < tiles; ++i) {
        const int k0 = k_lo + i * kKeys;
        __syncthreads();                                     // the last tile has been used
        if (tid < kKeys) rows[tid] = tid < k_hi - k0 ? cache_row(p.cache, n, k0 + tid) : -1;
        __syncthreads();
        for (int i = tid; i < kKeys * C4; i += kThreads) {
            const int key = i / C4, c = i % C4, row = rows[key];
            const size_t at = ((size_t)(row < 0 ? 0 : row) * p.cache.H_kv + hk) * C4 + c;
            const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(sk + key * L::kPitch + 4 * c) =
                row < 0 ? zero : reinterpret_cast<const float4 *>(kc)[at];
            *reinterpret_cast<float4 *>(sv + key * D + 4 * c) =
                row < 0 ? zero : reinterpret_cast<const float4 *>(vc)[at];
        }
        __syncthreads();
        float2 s2[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) s2[a][b] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < C4; ++c) {
            float4 q[4], k[4];
#pragma unroll
            for (int a = 0; a < 4; ++a) q[a] = *reinterpret_cast<const float4 *>(sq + (4 * ty + a) * L::kPitch + 4 * c);
#pragma unroll
            for (int b = 0; b < 4; ++b) k[b] = *reinterpret_cast<const float4 *>(sk + (tx + 16 * b) * L::kPitch + 4 * c);
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    s2[a][b] = fma2(make_float2(q[a].x, q[a].y), make_float2(k[b].x, k[b].y), s2[a][b]);
                    s2[a][b] = fma2(make_float2(q[a].z, q[a].w), make_float2(k[b].z, k[b].w), s2[a][b]);
                }
        }
        float s[4][4];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b) s[a][b] = s2[a][b].x + s2[a][b].y;
        score2<7>(reinterpret_cast<float(&)[16]>(s), p.score);
        __syncthreads();                                     // the keys have been used
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            float mx = m[a];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int key = tx + 16 * b;
                const bool live = key >= lo[a] - k0 && key < hi[a] - k0 && rows[key] >= 0;
                s[a][b] = live ? s[a][b] : -INFINITY;
                mx = fmaxf(mx, s[a][b]);
            }
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float shift = mx == -INFINITY ? 0.f : mx, f = ex2(m[a] - shift);
            m[a] = mx;
            l[a] *= f;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) o[a][d] = mul2(o[a][d], make_float2(f, f));
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const float w = ex2(s[a][b] - shift);
                l[a] += w;
                sp[(4 * ty + a) * (kKeys + 4) + tx + 16 * b] = w;
            }
        }
        __syncwarp();                                        // a half warp's rows are its own
#pragma unroll 2
        for (int k = 0; k < kKeys; k += 4) {
            float w[4][4];
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const float4 x = *reinterpret_cast<const float4 *>(sp + (4 * ty + a) * (kKeys + 4) + k);
                w[a][0] = x.x; w[a][1] = x.y; w[a][2] = x.z; w[a][3] = x.w;
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int d = 0; d < D / 64; ++d) {
                    const float4 v = *reinterpret_cast<const float4 *>(sv + (k + b) * D + 64 * d + 4 * tx);
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const float2 x = make_float2(w[a][b], w[a][b]);
                        o[a][2 * d] = fma2(x, make_float2(v.x, v.y), o[a][2 * d]);
                        o[a][2 * d + 1] = fma2(x, make_float2(v.z, v.w), o[a][2 * d + 1]);
                    }
                }
        }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        float sum = l[a];
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const long long r = r0 + 4 * ty + a;
        if (r >= r_end) continue;
        if (parts > 1) {                                     // this CTA's share, unnormalised
            const size_t part = ((size_t)block * p.splits + split) * kRows + 4 * ty + a;
            if (tx == 0) p.part_ml[part] = make_float2(m[a], sum);
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
                *reinterpret_cast<float4 *>(p.part_o + part * D + 64 * d + 4 * tx) =
                    make_float4(o[a][2 * d].x, o[a][2 * d].y, o[a][2 * d + 1].x, o[a][2 * d + 1].y);
            continue;
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const size_t at = row_at(r);
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * D + 64 * d + 4 * tx) =
                make_float4(o[a][2 * d].x * inv, o[a][2 * d].y * inv, o[a][2 * d + 1].x * inv, o[a][2 * d + 1].y * inv);
        if (tx == 0 && p.lse) p.lse[at] = sum > 0.f ? (m[a] + log2f(sum)) * kLn2 : -INFINITY;
    }
}

template <int D> PerDevice g_setup;

template <int D>
cudaError_t launch_dim(const AttnPrefillParams &p, cudaStream_t stream) {
    const cudaError_t e = g_setup<D>.ensure([] {
        return cudaFuncSetAttribute(attn_prefill_f32_kernel<D>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
    });
    if (e != cudaSuccess) return e;
    attn_prefill_f32_kernel<D><<<(unsigned)(p.blocks * p.splits), kThreads, Smem<D>::kBytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_f32(const AttnPrefillParams &p, int d, cudaStream_t stream) {
    return d == 128 ? launch_dim<128>(p, stream) : launch_dim<64>(p, stream);
}

}  // namespace gdn
