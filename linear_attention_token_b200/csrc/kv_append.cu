// gdn_kv_append (include/attn.h): keys and values into the paged cache, the rotation applied
// on the way, and the queries rotated beside them.
//
//   y[i]         = x[i] cos a - x[i + R/2] sin a
//   y[i + R/2]   = x[i + R/2] cos a + x[i] sin a,     a = position * inv_freq[i],  i < R/2
//
// Every element is read once and written once, so large calls are bound by HBM and small
// ones by the latency of the dependent loads (offsets -> page table -> store).  A warp takes a
// token (or a share of one): it issues its first loads, forms the token's sines and cosines in
// shared memory meanwhile, and uses them for every head.
#include <math.h>
#include <stdint.h>

#include "device_once.h"
#include "paged_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;           // largest rope_dims / 2
constexpr int kFewWarps = 32;          // below this many warps an SM a token is shared by several

struct AppendParams {
    PagedView cache;
    const unsigned char *k, *v, *q;
    unsigned char *q_out;
    long long k_stride, v_stride, q_stride;      // bytes between tokens
    const int32_t *cu, *pos0, *rope_pos;
    const float *inv_freq;
    long long T_total, T_seq;                    // T_seq: tokens per sequence when cu is null
    int num_seqs, H_q, half, n_axes;
    int sec[GDN_ROPE_MAX_AXES];
    bool interleaved;
    int split_shift;                             // 2^split_shift warps share a token
};

// Angle p * f in half turns of pi, in [-1, 1]: the product of a 33-bit position and a 24-bit
// frequency loses at most its last bits in a double, and is reduced there by a two-part 2 pi (Cody
// and Waite).
__device__ __forceinline__ float half_turns(long long p, float f) {
    const double x = (double)p * (double)f;
    const double n = rint(x * 0.15915494309189535);
    return (float)(fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, x)) * 0.3183098861837907);
}

__device__ __forceinline__ int axis_of(const AppendParams &p, int i) {
    if (p.n_axes == 1) return 0;
    if (p.interleaved) {
        const int a = i % p.n_axes;
        return i < p.n_axes * p.sec[a] ? a : 0;
    }
    return i < p.sec[0] ? 0 : i < p.sec[0] + p.sec[1] ? 1 : 2;
}

// Sequence of token t: the last n with cu[n] <= t (32 probes a step, so one step up to 32
// sequences, two up to 1024), or -1 past the last sequence.  The whole warp calls it.
__device__ int sequence_of(const int32_t *cu, int num_seqs, long long t) {
    const int lane = threadIdx.x & 31;
    if (t >= __ldg(cu + num_seqs)) return -1;
    int lo = 0, hi = num_seqs;                   // cu[lo] <= t < cu[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && __ldg(cu + at) <= t;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        hi = min(hi, lo + (c + 1) * step);
        lo += c * step;
    }
    return lo;
}

template <typename T> struct Pack;               // 16 bytes as fp32
template <> struct Pack<float> {
    static constexpr int kN = 4;
    __device__ static void get(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
    }
    __device__ static uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};
template <> struct Pack<__nv_bfloat16> {
    static constexpr int kN = 8;
    __device__ static void get(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ static uint4 put(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A token's work is `heads` rows of D / (2 VEC) items; an item is two 16-byte chunks of one row: a
// rotation pair, or two that pass through.  2^split_shift warps share a token's items; each forms
// the token's sines and cosines for itself, so warps never wait for one another.
// A lane has kBatch items (32 bytes each) in flight.  Many tokens: one, and 6 CTAs an SM (65,536
// tokens x 20 rows: 113 us, 92% of the measured copy rate; 8 CTAs, which spill, 116; two items with
// 5 CTAs 120, four with 3 130).  Few tokens: two, since nothing else hides the latency (3.5 against
// 4.1 us for 64 tokens x 48 rows).
template <typename T, int D, int kBatch>
__global__ void __launch_bounds__(kThreads, kBatch == 1 ? 6 : 5) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int VEC = Pack<T>::kN, IPR = D / (2 * VEC);     // items per row
    constexpr size_t ROW = (size_t)D * sizeof(T);
    __shared__ float2 trig_of[kThreads / 32][kMaxHalf];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long gw = (long long)blockIdx.x * (kThreads / 32) + warp;
    const long long t = gw >> p.split_shift;
    if (t >= p.T_total) return;
    float2 *trig = trig_of[warp];
    const int H_q = p.H_q, H_k = p.cache.H_kv, total = (H_q + 2 * H_k) * IPR;
    const int pairs = p.half / VEC;
    const int first = ((int)(gw & ((1 << p.split_shift) - 1)) << 5) + lane, step = 32 << p.split_shift;

    // chunks and place of item i: q heads, then keys, then values
    struct Item { int h, c0, c1; bool pair; };
    auto item = [&](int i) {
        Item x;
        x.h = i / IPR;
        const int j = i % IPR;
        const bool value = x.h >= H_q + H_k;
        x.pair = !value && j < pairs;
        x.c0 = x.pair ? j : 2 * j;                           // (past the pairs: 2 pairs + 2 (j - pairs))
        x.c1 = x.pair ? j + pairs : x.c0 + 1;
        return x;
    };
    uint4 a[kBatch], b[kBatch];
    auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * step;
            if (i >= total) continue;
            const Item x = item(i);
            const unsigned char *src = x.h < H_q         ? p.q + t * p.q_stride + x.h * ROW
                                       : x.h < H_q + H_k ? p.k + t * p.k_stride + (x.h - H_q) * ROW
                                                         : p.v + t * p.v_stride + (x.h - H_q - H_k) * ROW;
            a[u] = *reinterpret_cast<const uint4 *>(src + x.c0 * 16);
            b[u] = *reinterpret_cast<const uint4 *>(src + x.c1 * 16);
        }
    };
    load(first);                                             // in flight while the tables form

    int n;
    long long pos;
    if (p.cu) {
        n = sequence_of(p.cu, p.num_seqs, t);
        if (n < 0) return;                                   // behind the last sequence
        pos = t - __ldg(p.cu + n);
    } else {
        n = (int)(t / p.T_seq);
        pos = t - n * p.T_seq;
    }
    if (p.pos0) pos += __ldg(p.pos0 + n);
    const int row = cache_row(p.cache, n, pos);
    for (int i = lane; i < p.half; i += 32) {
        const long long at = p.rope_pos ? __ldg(p.rope_pos + axis_of(p, i) * p.T_total + t) : pos;
        float s, c;
        sincospif(half_turns(at, __ldg(p.inv_freq + i)), &s, &c);
        trig[i] = make_float2(c, s);
    }
    __syncwarp();
    for (int i0 = first; i0 < total;) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * step;
            if (i >= total) continue;
            const Item x = item(i);
            if (row < 0 && x.h >= H_q) continue;             // absent: keys and values go nowhere
            uint4 lo4 = a[u], hi4 = b[u];
            if (x.pair) {
                float lo[VEC], hi[VEC];
                Pack<T>::get(lo4, lo);
                Pack<T>::get(hi4, hi);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 cs = trig[x.c0 * VEC + e];
                    const float l = lo[e], h = hi[e];
                    lo[e] = l * cs.x - h * cs.y;
                    hi[e] = h * cs.x + l * cs.y;
                }
                lo4 = Pack<T>::put(lo);
                hi4 = Pack<T>::put(hi);
            }
            unsigned char *dst =
                x.h < H_q         ? p.q_out + ((size_t)t * H_q + x.h) * ROW
                : x.h < H_q + H_k ? p.cache.k + ((size_t)row * H_k + (x.h - H_q)) * ROW
                                  : p.cache.v + ((size_t)row * H_k + (x.h - H_q - H_k)) * ROW;
            *reinterpret_cast<uint4 *>(dst + x.c0 * 16) = lo4;
            *reinterpret_cast<uint4 *>(dst + x.c1 * 16) = hi4;
        }
        i0 += kBatch * step;
        load(i0);
    }
}

template <typename T, int D>
cudaError_t launch_typed(AppendParams p, int sms, cudaStream_t stream) {
    // warps per token: enough that a few tokens still spread over the SMs, no more than have items
    const int items = (p.H_q + 2 * p.cache.H_kv) * D / (2 * Pack<T>::kN);
    while (p.split_shift < 3 && (p.T_total << p.split_shift) < (long long)sms * kFewWarps &&
           (32 << p.split_shift) < items)
        ++p.split_shift;
    const long long warps = p.T_total << p.split_shift;
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    if (p.split_shift == 0)
        kv_append_kernel<T, D, 1><<<grid, kThreads, 0, stream>>>(p);
    else
        kv_append_kernel<T, D, 2><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const gdn_paged_kv &kv, const void *k, const void *v, const void *q,
                             void *q_out, long long k_stride, long long v_stride,
                             long long q_stride, const int32_t *cu, const int32_t *pos0,
                             int num_seqs, long long T_total, int H_q, const float *inv_freq,
                             int rope_dims, const int32_t *rope_pos, const int32_t *sections,
                             int n_axes, bool interleaved, int sms, cudaStream_t stream) {
    const int esize = kv.dtype == GDN_BF16 ? 2 : 4;
    AppendParams p = {};
    p.cache = paged_view(kv);
    p.k = static_cast<const unsigned char *>(k);
    p.v = static_cast<const unsigned char *>(v);
    p.q = static_cast<const unsigned char *>(q);
    p.q_out = static_cast<unsigned char *>(q_out);
    p.k_stride = k_stride * esize;
    p.v_stride = v_stride * esize;
    p.q_stride = q_stride * esize;
    p.cu = cu;
    p.pos0 = pos0;
    p.rope_pos = rope_pos;
    p.inv_freq = inv_freq;
    p.T_total = T_total;
    p.T_seq = cu ? 0 : T_total / num_seqs;
    p.num_seqs = num_seqs;
    p.H_q = q ? H_q : 0;
    p.half = rope_dims / 2;
    p.n_axes = n_axes;
    for (int a = 0; a < GDN_ROPE_MAX_AXES; ++a) p.sec[a] = sections && a < n_axes ? sections[a] : 0;
    p.interleaved = interleaved;
    if (kv.dtype == GDN_BF16)
        return kv.d == 128 ? launch_typed<__nv_bfloat16, 128>(p, sms, stream)
                           : launch_typed<__nv_bfloat16, 64>(p, sms, stream);
    return kv.d == 128 ? launch_typed<float, 128>(p, sms, stream) : launch_typed<float, 64>(p, sms, stream);
}

}  // namespace gdn
