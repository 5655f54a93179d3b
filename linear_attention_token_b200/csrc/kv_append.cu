// gdn_kv_append (include/attn.h): keys and values into the paged cache, the rotation applied
// on the way, and the queries rotated beside them.
//
//   y[i]         = x[i] cos a - x[i + R/2] sin a
//   y[i + R/2]   = x[i + R/2] cos a + x[i] sin a,     a = position * inv_freq[i],  i < R/2
//
// Every element is read once and written once, so large calls are bound by HBM and small
// ones by the latency of the dependent loads (offsets -> page table -> store).  A CTA takes
// kTokens tokens; their angles' sines and cosines are formed once in shared memory and used
// by every head, and the x loads are issued before that table is ready.
#include <math.h>
#include <stdint.h>

#include "device_once.h"
#include "paged_kv.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;          // one warp finds one token's sequence and row
constexpr int kMaxHalf = 64;           // largest rope_dims / 2

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
};

// Angle p * f reduced to [-pi, pi] in double precision (a two-part 2 pi; Cody and Waite).  The
// product of a 32-bit position and a 24-bit frequency loses at most its last bits in a double.
__device__ __forceinline__ float turn(int p, float f) {
    const double x = (double)p * (double)f;
    const double n = rint(x * 0.15915494309189535);
    return (float)fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586, x));
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

// One item is two 16-byte chunks of one head: a rotation pair, or two that pass through.
template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int VEC = Pack<T>::kN, IPR = D / (2 * VEC);     // items per head
    constexpr int BATCH = 4;                                  // items in flight per thread
    __shared__ float2 trig[TOK][kMaxHalf];
    __shared__ int row_of[TOK];                               // cache row, -1 absent, -2 no token
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long t0 = (long long)blockIdx.x * TOK;
    const int heads = p.H_q + 2 * p.cache.H_kv;
    const int per_token = heads * IPR, total = per_token * TOK;
    const int pairs = p.half / VEC;

    if (warp < TOK) {
        const long long t = t0 + warp;
        int n = -1;
        long long pos = 0;
        if (t < p.T_total) {
            n = p.cu ? sequence_of(p.cu, p.num_seqs, t) : (int)(t / p.T_seq);
            if (n >= 0)
                pos = t - (p.cu ? (long long)__ldg(p.cu + n) : n * p.T_seq) +
                      (p.pos0 ? __ldg(p.pos0 + n) : 0);
        }
        if (lane == 0) row_of[warp] = n < 0 ? -2 : cache_row(p.cache, n, pos);
        if (n >= 0)
            for (int i = lane; i < p.half; i += 32) {
                const int at = p.rope_pos ? __ldg(p.rope_pos + axis_of(p, i) * p.T_total + t)
                                          : (int)pos;
                float s, c;
                sincosf(turn(at, __ldg(p.inv_freq + i)), &s, &c);
                trig[warp][i] = make_float2(c, s);
            }
    }
    for (int i0 = tid; i0 - tid < total; i0 += kThreads * BATCH) {       // uniform over the CTA
        uint4 a[BATCH], b[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int i = i0 + u * kThreads;
            const int tok = i / per_token, r = i - tok * per_token, h = r / IPR, j = r - h * IPR;
            if (i >= total || t0 + tok >= p.T_total) continue;
            const bool value = h >= p.H_q + p.cache.H_kv;
            const bool pair = !value && j < pairs;
            const unsigned char *src =
                value ? p.v + (t0 + tok) * p.v_stride + (size_t)(h - p.H_q - p.cache.H_kv) * D * sizeof(T)
                : h >= p.H_q ? p.k + (t0 + tok) * p.k_stride + (size_t)(h - p.H_q) * D * sizeof(T)
                             : p.q + (t0 + tok) * p.q_stride + (size_t)h * D * sizeof(T);
            const int c0 = pair ? j : value ? 2 * j : 2 * pairs + 2 * (j - pairs);
            const int c1 = pair ? j + pairs : c0 + 1;
            a[u] = *reinterpret_cast<const uint4 *>(src + c0 * 16);
            b[u] = *reinterpret_cast<const uint4 *>(src + c1 * 16);
        }
        if (i0 == tid) __syncthreads();                     // the tables; the loads are in flight
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int i = i0 + u * kThreads;
            if (i >= total) continue;
            const int tok = i / per_token, r = i - tok * per_token, h = r / IPR, j = r - h * IPR;
            const int row = row_of[tok];
            if (row == -2 || (row < 0 && h >= p.H_q)) continue;
            const bool value = h >= p.H_q + p.cache.H_kv;
            const bool pair = !value && j < pairs;
            if (pair) {
                float x[VEC], y[VEC];
                Pack<T>::get(a[u], x);
                Pack<T>::get(b[u], y);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float2 cs = trig[tok][j * VEC + e];
                    const float lo = x[e], hi = y[e];
                    x[e] = lo * cs.x - hi * cs.y;
                    y[e] = hi * cs.x + lo * cs.y;
                }
                a[u] = Pack<T>::put(x);
                b[u] = Pack<T>::put(y);
            }
            const int c0 = pair ? j : value ? 2 * j : 2 * pairs + 2 * (j - pairs);
            const int c1 = pair ? j + pairs : c0 + 1;
            const size_t head = (size_t)D * sizeof(T);
            unsigned char *dst =
                value ? p.cache.v + ((size_t)row * p.cache.H_kv + (h - p.H_q - p.cache.H_kv)) * head
                : h >= p.H_q ? p.cache.k + ((size_t)row * p.cache.H_kv + (h - p.H_q)) * head
                             : p.q_out + ((size_t)(t0 + tok) * p.H_q + h) * head;
            *reinterpret_cast<uint4 *>(dst + c0 * 16) = a[u];
            *reinterpret_cast<uint4 *>(dst + c1 * 16) = b[u];
        }
    }
}

template <typename T, int D>
cudaError_t launch_typed(const AppendParams &p, cudaStream_t stream) {
    if (p.T_total < 2048)
        kv_append_kernel<T, D, 1><<<(unsigned)p.T_total, kThreads, 0, stream>>>(p);
    else
        kv_append_kernel<T, D, kMaxTokens>
            <<<(unsigned)((p.T_total + kMaxTokens - 1) / kMaxTokens), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const gdn_paged_kv &kv, const void *k, const void *v, const void *q,
                             void *q_out, long long k_stride, long long v_stride,
                             long long q_stride, const int32_t *cu, const int32_t *pos0,
                             int num_seqs, long long T_total, int H_q, const float *inv_freq,
                             int rope_dims, const int32_t *rope_pos, const int32_t *sections,
                             int n_axes, bool interleaved, cudaStream_t stream) {
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
        return kv.d == 128 ? launch_typed<__nv_bfloat16, 128>(p, stream)
                           : launch_typed<__nv_bfloat16, 64>(p, stream);
    return kv.d == 128 ? launch_typed<float, 128>(p, stream) : launch_typed<float, 64>(p, stream);
}

}  // namespace gdn
