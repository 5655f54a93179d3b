// gdn_attn_prefill (include/attn.h): how a call is cut, the split of long contexts over CTAs when there
// are few query rows, and the join of the parts.
//
// A block of query rows (256 in bf16, 64 in fp32) walks all the tokens it sees in one CTA; a call
// with fewer blocks than the SMs run at once would leave the others idle for as long as that takes
// (64 new tokens behind 100,000 cached ones: 4 CTAs).  Such a call gives each block as many CTAs as
// fill the SMs, each a stretch of the K / V tiles, and joins their maxima, sums and outputs with a
// second kernel.  A CTA takes at least kSplitTiles tiles: below that the fp32 parts and the second
// launch cost more than the shorter walk saves.  The host knows no lengths, only what the page
// table can hold: a block that turns out short is run whole by its first CTA, and the join passes
// over it (a short prompt behind a wide table: 64 tokens x 16 x 2 heads 11.4 us for 10.1, 333 15.1 for 13.5,
// 700 20.8 for 19.8, and up to 20 MB of workspace).
#include <math.h>
#include <stdint.h>

#include "attn_prefill.cuh"
#include "device_once.h"

namespace gdn {

cudaError_t launch_attn_prefill_bf16(const AttnPrefillParams &p, const gdn_paged_kv &kv, cudaStream_t stream);
cudaError_t launch_attn_prefill_f32(const AttnPrefillParams &p, int d, cudaStream_t stream);

namespace {

constexpr int kMaxSplits = 64;

// Row r of block (x, r) from its parts: out = sum_i e^{m_i - m} O_i / sum_i e^{m_i - m} l_i.  A warp
// takes a row.
template <typename E, int D>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(const __grid_constant__ AttnPrefillParams p,
                                                                int rows) {
    constexpr int V = D / 32;
    pdl_wait();
    const SplitBlock b = p.split_blocks[blockIdx.x];
    const int r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int token = (b.row0 + r) / max(b.pack, 1);
    if (b.parts < 2 || token >= b.len) return;
    const size_t at0 = (size_t)blockIdx.x * p.splits * rows + r;
    // a lane weighs a part (or two: there are at most kMaxSplits), and the outputs, which do not wait for
    // the weights, come in several at a time
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 ml0 = lane < b.parts ? p.part_ml[at0 + (size_t)lane * rows] : none;
    const float2 ml1 = lane + 32 < b.parts ? p.part_ml[at0 + (size_t)(lane + 32) * rows] : none;
    float m = fmaxf(ml0.x, ml1.x);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float shift = m == -INFINITY ? 0.f : m;
    // a part without tokens (l = 0) wrote no outputs: it is not read
    const float f0 = ml0.y > 0.f ? ex2(ml0.x - shift) : 0.f, f1 = ml1.y > 0.f ? ex2(ml1.x - shift) : 0.f;
    const float l = warp_sum(ml0.y * f0 + ml1.y * f1);
    const uint32_t some[2] = {__ballot_sync(0xffffffffu, ml0.y > 0.f), __ballot_sync(0xffffffffu, ml1.y > 0.f)};
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll 8
    for (int i = 0; i < b.parts; ++i) {
        if (!((some[i >> 5] >> (i & 31)) & 1)) continue;
        const float f = __shfl_sync(0xffffffffu, i < 32 ? f0 : f1, i & 31);
        const float *src = p.part_o + (at0 + (size_t)i * rows) * D + lane * V;
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(src);
            o[0] = fmaf(x.x, f, o[0]);
            o[1] = fmaf(x.y, f, o[1]);
            o[2] = fmaf(x.z, f, o[2]);
            o[3] = fmaf(x.w, f, o[3]);
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(src);
            o[0] = fmaf(x.x, f, o[0]);
            o[1] = fmaf(x.y, f, o[1]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const size_t rh = (size_t)(b.first + token) * p.H_q + b.h0 + (b.row0 + r) % b.pack;
    E *dst = static_cast<E *>(p.out) + rh * D + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        if constexpr (sizeof(E) == 2)
            *reinterpret_cast<uint32_t *>(dst + e) = pack2(o[e] * inv, o[e + 1] * inv);
        else
            *reinterpret_cast<float2 *>(dst + e) = make_float2(o[e] * inv, o[e + 1] * inv);
    }
    if (lane == 0 && p.lse) p.lse[rh] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

struct Shape {
    int pack_shift, rows, splits;          // heads packed into a row tile (bf16), rows of a block
    long long blocks;                      // (block, head) pairs, at most
    size_t bytes() const { return kErrorBytes + table_bytes() + (size_t)blocks * splits * rows * row_bytes; }
    size_t table_bytes() const { return ((size_t)blocks * sizeof(SplitBlock) + 255) / 256 * 256; }
    size_t row_bytes;                      // of a part
};
Shape prefill_shape(const gdn_paged_kv &kv, bool varlen, int N, long long T_total, int H_q, int sms) {
    Shape s = {};
    const int G = H_q / kv.H_kv;
    // one block of a sequence may be part full (packed tokens that fill their blocks are counted one block a
    // sequence too many, whose CTAs leave at once: 64 x 16 x 2 heads behind 100,000 runs on 96 of 148 SMs, 82 us)
    auto bound = [&](long long total, long long size) {
        return varlen ? total / size + N : (total / N + size - 1) / size * N;
    };
    const bool f32 = kv.dtype == GDN_F32;
    if (f32) {
        s.rows = kF32Rows;
        s.blocks = varlen ? bound(T_total * G, s.rows) : (T_total / N * G + s.rows - 1) / s.rows * N;
        s.blocks *= kv.H_kv;
    } else {
        // the largest power of two, up to 16, that divides the group
        while (s.pack_shift < 4 && G % (2 << s.pack_shift) == 0) ++s.pack_shift;
        s.rows = kPrefillRows;
        s.blocks = bound(T_total, s.rows >> s.pack_shift) * kv.H_kv * (G >> s.pack_shift);
    }
    s.row_bytes = sizeof(float2) + kv.d * sizeof(float);
    const long long slots = (f32 ? 2LL : 1LL) * sms;          // CTAs that run at once
    const long long tiles = (long long)kv.max_pages * kv.page_size / (f32 ? kF32Keys : kPrefillTile);
    long long splits = s.blocks > 0 ? slots / s.blocks : 1;
    if (splits > tiles / kSplitTiles) splits = tiles / kSplitTiles;
    s.splits = splits < 1 ? 1 : splits > kMaxSplits ? kMaxSplits : (int)splits;
    return s;
}

template <typename E, int D>
cudaError_t launch_join(const AttnPrefillParams &p, int rows, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.blocks, (unsigned)(rows / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_prefill_join_kernel<E, D>, p, rows);
}

}  // namespace

size_t attn_prefill_workspace_bytes(const gdn_paged_kv &kv, bool varlen, int N, long long T_total, int H_q,
                                    int sms) {
    const Shape s = prefill_shape(kv, varlen, N, T_total, H_q, sms);
    return s.splits > 1 ? s.bytes() : kErrorBytes;
}

int attn_prefill_splits(const gdn_paged_kv &kv, int N, long long T_total, int H_q, int sms) {
    return prefill_shape(kv, false, N, T_total, H_q, sms).splits;
}

cudaError_t launch_attn_prefill(const gdn_paged_kv &kv, const void *q, const int32_t *cu,
                                const int32_t *pos0, const int32_t *prefix, void *out, float *lse,
                                int N, long long T_total, int H_q, float scale, float cap, int window,
                                void *workspace, size_t workspace_bytes, int sms, uint32_t budget,
                                cudaStream_t stream) {
    Shape s = prefill_shape(kv, cu != nullptr, N, T_total, H_q, sms);
    if (s.splits > 1 && (!workspace || workspace_bytes < s.bytes())) s.splits = 1;
    if (s.blocks * s.splits > INT32_MAX) return cudaErrorInvalidValue;
    AttnPrefillParams p = {};
    p.cache = paged_view(kv);
    p.q = q;
    p.out = out;
    p.lse = lse;
    p.cu = cu;
    p.pos0 = pos0;
    p.prefix = prefix;
    p.T_total = T_total;
    p.T_seq = cu ? 0 : T_total / N;
    p.N = N;
    p.H_q = H_q;
    p.G = H_q / kv.H_kv;
    p.window = window;
    p.pack_shift = s.pack_shift;
    p.score = scoring(scale, cap);
    // The bf16 kernel's polynomials for capped scores carry the factors cap2 k^(2i+1), k = scale / cap, in
    // their coefficients.  Degree 5 (|y| <= 1; degree 3 for |y| <= 1/2) serves where the first and the last
    // of these, and so all between, are inside fp32 with room for a coefficient below and a sum above
    // (2^-124: a coefficient that is no longer normal is off by 2^-26 of the whole at most); else degree 2
    // (|y| <= 1/8; caps from 390 at a scale of 0.09), else none.
    const double k = fabs((double)p.score.mul), cap2 = p.score.cap2;
    auto inside = [&](int degree) {
        const double first = k * cap2, last = first * pow(k, 2 * degree);
        return fmin(first, last) >= 0x1p-124 && fmax(first, last) <= 0x1p120 && k >= 0x1p-60 && k <= 0x1p60;
    };
    const bool all = inside(5);
    p.near_at = all ? 1.f : inside(2) ? 0.125f : -1.f;
    p.nearer_at = all ? 0.5f : -1.f;
    p.err = static_cast<DeviceError *>(workspace);
    p.budget = budget;
    p.blocks = s.blocks;
    p.splits = s.splits;
    if (s.splits > 1) {
        unsigned char *at = static_cast<unsigned char *>(workspace) + kErrorBytes;
        p.split_blocks = reinterpret_cast<SplitBlock *>(at);
        p.part_ml = reinterpret_cast<float2 *>(at + s.table_bytes());
        p.part_o = reinterpret_cast<float *>(p.part_ml + (size_t)s.blocks * s.splits * s.rows);
    }
    const bool f32 = kv.dtype == GDN_F32;
    const cudaError_t e = f32 ? launch_attn_prefill_f32(p, kv.d, stream) : launch_attn_prefill_bf16(p, kv, stream);
    if (e != cudaSuccess || s.splits == 1) return e;
    if (f32)
        return kv.d == 128 ? launch_join<float, 128>(p, s.rows, stream) : launch_join<float, 64>(p, s.rows, stream);
    return kv.d == 128 ? launch_join<__nv_bfloat16, 128>(p, s.rows, stream)
                       : launch_join<__nv_bfloat16, 64>(p, s.rows, stream);
}

}  // namespace gdn
