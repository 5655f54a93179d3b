// Exponentials and capped scores of the attention kernels.  Scores are kept in base-2 units: log2(e)
// times the scaled, capped score.
#pragma once

#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Two fp32 lanes per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// tanh(y) = y R(y^2), R fitted to the least largest relative error: of degree 7 for |y| <= 1 (4.2e-9, a
// fourteenth of 2^-24), of degree 5 for |y| <= 1 (5.9e-7, ten times 2^-24), of degree 3 for |y| <= 1/2
// (5.5e-7); of degree 2 the series, for |y| <= 1/8 (2.1e-7).  Degree 7 serves fp32, whose capped scores are
// then right to roundings (it costs 1% with eight rows or in prompts, with degree 5 before); bf16 takes the
// shorter ones: a capped score there, and so lse, is off by up to 2^-20 of itself, far less than the
// weights' rounding to bf16.
template <int DEG>
__device__ constexpr float tanh_r(int i) {
    constexpr float c7[8] = {1.f,           -0.3333327868f, 0.1333215967f, -0.0538709128f,
                             0.0214648203f, -0.0079174447f, 0.0022822296f, -0.0003533455f};
    constexpr float c5[6] = {0.9999994136f, -0.3332904242f, 0.1328143402f,
                             -0.0516056755f, 0.0167431149f, -0.0030670597f};
    constexpr float c3[4] = {0.9999994636f, -0.3332631886f, 0.1319029629f, -0.0444022268f};
    constexpr float c2[3] = {1.f, -1.f / 3.f, 2.f / 15.f};
    return DEG == 7 ? c7[i & 7] : DEG == 5 ? c5[i % 6] : DEG == 3 ? c3[i & 3] : c2[i % 3];
}

// What turns a dot product into a score: scale alone, or scale and cap.
struct Scoring {
    float mul;                             // no cap: scale log2 e; cap: scale / cap
    float cap2;                            // cap log2 e; 0: no cap
};
inline Scoring scoring(float scale, float cap) {
    Scoring s;
    s.mul = cap > 0.f ? scale / cap : scale * kLog2e;
    // (a quotient past fp32 becomes its largest number, since infinity times a zero score is none; any
    // other score is the cap then either way)
    if (cap > 0.f) s.mul = fminf(fmaxf(s.mul, -3.402823466e38f), 3.402823466e38f);
    s.cap2 = cap * kLog2e;
    return s;
}
// cap2 tanh(y) for |y| <= 1 (DEG 7 or 5) or 1/2 (3), by the polynomial: off by its fit and 5 2^-24
template <int DEG> __device__ __forceinline__ float2 capped_near2(float2 y, float cap2) {
    const float2 t = mul2(y, y);
    float2 r = make_float2(tanh_r<DEG>(DEG), tanh_r<DEG>(DEG));
#pragma unroll
    for (int i = DEG - 1; i >= 0; --i) r = fma2(r, t, make_float2(tanh_r<DEG>(i), tanh_r<DEG>(i)));
    return mul2(mul2(y, r), make_float2(cap2, cap2));
}
// cap2 tanh(y) for any y: beyond 1/2 (DEG 3) or 1 (DEG 7) as 1 - 2 / (1 + e^{2y}), which is off by a few
// 2^-24 of the cap and so would leave nothing of a score far below a large one
template <int DEG> __device__ __forceinline__ float2 capped2(float2 y, float cap2) {
    constexpr float kNear = DEG == 3 ? 0.5f : 1.f;
    const float2 near = capped_near2<DEG>(y, cap2);
    const float2 x = mul2(y, make_float2(2.f * kLog2e, 2.f * kLog2e));
    const float2 e = add2(make_float2(ex2(x.x), ex2(x.y)), make_float2(1.f, 1.f));
    const float2 far = fma2(make_float2(__fdividef(2.f, e.x), __fdividef(2.f, e.y)), make_float2(-cap2, -cap2),
                            make_float2(cap2, cap2));
    return make_float2(fabsf(y.x) <= kNear ? near.x : far.x, fabsf(y.y) <= kNear ? near.y : far.y);
}
// N dot products of each lane to scores, in place; the warp takes the polynomial of degree DEG (7 or 5) when
// none of its scores passes the cap.  The whole warp calls it.
template <int DEG, int N>
__device__ __forceinline__ void score2(float (&x)[N], const Scoring &s) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= s.mul;
    if (s.cap2 == 0.f) return;
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) far = fmaxf(far, fabsf(x[i]));
    auto cap_all = [&](auto &&cap) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 c = cap(make_float2(x[i], i + 1 < N ? x[i + 1] : 0.f));
            x[i] = c.x;
            if (i + 1 < N) x[i + 1] = c.y;
        }
    };
    if (__any_sync(0xffffffffu, far > 1.f)) cap_all([&](float2 y) { return capped2<DEG == 7 ? 7 : 3>(y, s.cap2); });
    else cap_all([&](float2 y) { return capped_near2<DEG>(y, s.cap2); });
}

}  // namespace gdn
